"""Rotated pairs with elements that are not finite in the latent cache's append: NaN where the products' sum is NaN,
an infinity saturated, and the neighbours' pairs untouched."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("position", [0, 5, 70001])
def test_rotated_pairs(interleaved, position):
    import torch
    import mixed_attention_quantized_gb300 as mq
    inf, nan = float("inf"), float("nan")
    pairs = {1: (inf, 2.0), 4: (-3.0, -inf), 9: (inf, inf), 12: (inf, -inf), 20: (nan, 1.0), 31: (0.0, nan)}
    x = np.random.default_rng(5).standard_normal(64).astype(np.float32)
    places = [(2 * p, 2 * p + 1) if interleaved else (p, p + 32) for p in range(32)]
    for p, (a, b) in pairs.items():
        x[places[p][0]], x[places[p][1]] = a, b
    rope = mq.Rope(64, layout=int(interleaved))
    f = np.array(rope.info()["frequencies"])
    cache = mq.LatentCache.allocate(1)
    k = torch.from_numpy(x).half().cuda()[None]
    q = k.expand(1, 64).reshape(1, 1, 64).clone()
    i = torch.tensor([position], dtype=torch.int32, device="cuda")
    q_out = mq.latent_append(cache, rope, q, torch.zeros(1, 512, dtype=torch.float16, device="cuda"), k, i, i * 0)
    x = k[0].double().cpu().numpy()
    for got in (cache.data[0, 0, 512:], q_out[0, 0]):
        got = got.double().cpu().numpy()
        for p, (u, v) in enumerate(places):
            c, s = np.cos(position * f[p]), np.sin(position * f[p])
            with np.errstate(invalid="ignore"):
                want = np.array([x[u] * c - x[v] * s, x[v] * c + x[u] * s])
            y = got[[u, v]]
            if p not in pairs:
                bound = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2.0 ** -20 * (abs(x[u]) + abs(x[v]))
                assert (np.abs(y - want) <= bound).all()
                continue
            for a, b in zip(y, want):
                assert np.isnan(a) if np.isnan(b) else a == np.sign(b) * 65504, (p, y, want)

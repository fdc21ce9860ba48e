"""Lists with fewer entries than rows are refused before the library reads past their ends (no GPU)."""
import pytest

import mixed_attention_quantized_gb300 as mq

torch = pytest.importorskip("torch")

KINDS, SEQS, OFFS = [0, 0], [20, 30], [19, 29]
SHORT = [(KINDS[:1], SEQS, OFFS), (KINDS, SEQS, OFFS[:1]), ([], SEQS, OFFS)]


def _latent():
    cache = mq.LatentCache(4)
    cache.data = torch.zeros(4, 32, 576, dtype=torch.float16)
    return cache


@pytest.mark.parametrize("kinds,seqs,offs", SHORT)
def test_paged_plans_and_calls(kinds, seqs, offs):
    cache = mq.KVCache.allocate(4, 2, 64, mq.Q8_0, mq.Q8_0, device="cpu")
    q, pt = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: mq.Plan(cache, 4, kinds, seqs, offs, 1), lambda: mq.workspace_bytes(cache, 4, kinds, seqs, offs, 1),
                 lambda: mq.mixed_attention(cache, q, pt, seqs, offs, kinds),
                 lambda: mq.mixed_attention_noalloc(cache, q, pt, seqs, offs, kinds, o=q)):
        with pytest.raises(ValueError, match="entries"):
            call()


@pytest.mark.parametrize("kinds,seqs,offs", SHORT)
def test_latent_plans(kinds, seqs, offs):
    with pytest.raises(ValueError, match="entries"):
        mq.LatentPlan(_latent(), 4, kinds, seqs, offs, 1, 0.07)
    if len(offs) < len(seqs):
        with pytest.raises(ValueError, match="entries"):
            mq.ExpandedPlan(4, seqs, offs, 0.07)


def test_updates():
    for cls, args in ((mq.Plan, ([0], SEQS, OFFS, 1)), (mq.LatentPlan, ([0], SEQS, OFFS, 1)), (mq.ExpandedPlan, (SEQS, [0]))):
        plan = cls.__new__(cls)
        plan._lib, plan._handle = mq.load(), None
        with pytest.raises(ValueError, match="entries"):
            plan.update(*args)

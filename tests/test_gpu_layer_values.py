"""Attention over the 8-bit cache (include/lora_layer.h) where the sizes of values, keys and queries differ much, and where
slots that nobody sees hold anything.  The reference and its tolerances are those of test_gpu_layer.py."""
import pytest
import torch

from test_gpu_layer import TYPES, Step, ids

pytestmark = pytest.mark.gpu

# kernels for few rows and for many, sequences that are cut among them
SEQS = [[(1, 400), (3, 330)], [(100, 400)], [(2, 5000)], [(60, 3000)]]


def scale_keys(step, which, s, keys, factor):
    """Keys of sequence s in their pages: the scales `which` (ks or vs) times factor."""
    j = torch.as_tensor(keys)
    page = step.pages[s].long()[j // step.page]
    t = getattr(step, which)
    t[page, :, j % step.page] = t[page, :, j % step.page] * factor


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 128, 200, 256])
def test_attention_of_single_tokens_among_drafts(d, dtype):
    """Sequences of one row block in a launch for two, with and without masked tiles."""
    for window, sinks in ((0, 0), (60, 1)):
        Step([(8, 8 + 7 * i) for i in range(3)] + [(1, x) for x in (90, 1, 64, 63, 200)], 4, 1, d, 16, dtype, window=window,
             sinks=sinks).check()
        Step([(5 + i % 4, 8 + 5 * i) for i in range(20)] + [(1, 90), (1, 64), (2, 300)], 8, 2, d, 16, dtype, window=window,
             sinks=sinks).check()


# ------------------------------------------------- tiles whose values are small --
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("factor", [0.0, 2.0 ** -26, 2.0 ** -40], ids=["zero", "2^-26", "2^-40"])
def test_attention_small_values_keep_their_weight(factor, d, dtype):
    """Whole tiles of keys whose values are zero or tiny, first, in the middle or last: they take their share of the softmax
    all the same."""
    for seqs in SEQS[:2]:
        for lo, hi in ((0, 128), (128, 256), (192, 400), (64, 400)):
            step = Step(seqs, 4, 2, d, 16, dtype)
            for s, (_, x) in enumerate(seqs):
                scale_keys(step, "vs", s, range(lo, min(hi, x)), factor)
            step.check()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("factor", [0.0, 2.0 ** -40], ids=["zero", "2^-40"])
def test_attention_small_values_in_cut_units(factor, d, dtype):
    for seqs in SEQS[2:]:
        x = seqs[0][1]
        for lo, hi in ((0, x // 2), (x // 2, x), (64, x - 64)):
            step = Step(seqs, 4, 2, d, 16, dtype)
            scale_keys(step, "vs", 0, range(lo, hi), factor)
            step.check()
            assert sum(step.plan[:24].view(torch.int32).cpu().tolist()[4:6]) == 1


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 128, 200])
def test_attention_a_last_key_of_value_zero(d, dtype):
    """Alone in its tile, with a score above all others."""
    for n in (1, 100):
        step = Step([(n, 129)], 4, 2, d, 16, dtype)
        page = int(step.pages[0, 8])
        step.k[page, :, 0, :d] = (step.q[-1, ::2].float() * 40).round().clamp(-127, 127).to(torch.int8)
        step.vs[page] = 0.0
        step.check()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_attention_values_that_shrink_from_tile_to_tile(dtype):
    """Each tile's values 2^-3 of those of the one before it, or 2^3."""
    for seqs in SEQS[:2]:
        for factor in (0.125, 8.0):
            step = Step(seqs, 4, 2, 128, 16, dtype)
            for s, (_, x) in enumerate(seqs):
                for t in range(0, x, 64):
                    scale_keys(step, "vs", s, range(t, min(t + 64, x)), factor ** (t // 64))
            step.check()

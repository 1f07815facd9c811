"""Attention over the 8-bit cache (include/lora_layer.h) where the sizes of values, keys and queries differ much, and where
slots that nobody sees hold anything.  The reference and its tolerances are those of test_gpu_layer.py."""
import pytest
import torch

import rank_sgmv_bgmv_amd as L
from test_gpu_layer import H, TYPES, V, Step, branches, gen, half, ids, same

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


# ------------------------------------------------------ slots that nobody sees --
ODD = [1e30, 1e-30, float("inf"), -float("inf"), -3.0, float("nan")]


def fill_unseen(step, value, pages=True):
    """Scales of keys that no query of the batch sees, in the pages of those that are seen and (pages) in the whole of the
    others; what is in them is what a former request left."""
    seen = torch.zeros(step.k.shape[0], step.page, dtype=torch.bool)
    for s, (n, x) in enumerate(step.seqs):
        any_row = torch.stack([step.sees(s, i) for i in range(n)]).any(0)
        j = torch.arange(x)[any_row]
        seen[step.pages[s].long()[j // step.page], j % step.page] = True
    if not pages:
        seen |= ~seen.any(1, keepdim=True)
    for t in (step.ks, step.vs):
        t.transpose(1, 2)[~seen] = value


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("value", ODD, ids=str)
@pytest.mark.parametrize("d", [64, 128, 200])
def test_attention_slots_behind_a_sequence_may_hold_anything(d, value, dtype):
    """Never written, or left by a former request: the same bits as with ordinary scales there."""
    for seqs in ([(1, 50), (3, 17), (2, 129), (1, 16)], [(100, 250), (40, 41)], [(2, 5003)], [(60, 3001)]):
        step = Step(seqs, 4, 2, d, 16, dtype)
        clean = step.check()
        fill_unseen(step, value)
        assert same(step.run(), clean)
        step = Step(seqs, 4, 2, d, 64, dtype)
        clean = step.run()
        fill_unseen(step, value)
        assert same(step.run(), clean)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("value", ODD, ids=str)
@pytest.mark.parametrize("window, sinks", [(100, 5), (37, 0), (1, 70), (130, 129)])
def test_attention_slots_before_a_window_may_hold_anything(window, sinks, value, dtype):
    for seqs in ([(1, 1000), (1, 700), (2, 333)], [(20, 900), (50, 401)], [(130, 700)]):
        for page in (16, 64):
            step = Step(seqs, 4, 2, 64, page, dtype, window=window, sinks=sinks)
            clean = step.check()
            fill_unseen(step, value)
            assert same(step.run(), clean)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("value", ODD, ids=str)
def test_attention_pages_that_are_not_seen_may_be_any_page(value, dtype):
    """Entries of the page table that no query sees name a page of scales that would do harm."""
    for seqs in ([(1, 1000), (2, 333)], [(20, 900), (50, 401)]):
        step = Step(seqs, 4, 2, 64, 16, dtype, window=100, sinks=5)
        clean = step.check()
        free = sorted(set(range(step.k.shape[0])) - set(step.pages.flatten().tolist()))[0]
        step.ks[free] = step.vs[free] = value
        for s, (n, x) in enumerate(seqs):
            live = torch.zeros(step.pages.shape[1], dtype=torch.bool)
            live[0] = True
            live[(x - n - 100 + 1) // 16:-(-x // 16)] = True
            step.pages[s, ~live] = free
        assert same(step.run(), clean)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("value", ODD[2:], ids=str)
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_attention_a_key_without_a_finite_scale(which, value, dtype):
    """Scales that are no scales make the rows NaN that see the key, in its cache head, and no others."""
    for seqs in ([(4, 150)], [(100, 150)]):
        step = Step(seqs, 4, 2, 64, 16, dtype)
        n, x = seqs[0]
        getattr(step, which)[int(step.pages[0, (x - 2) // 16]), 1, (x - 2) % 16] = value
        got = step.run()
        want = torch.zeros(n, 4, dtype=torch.bool)
        want[n - 2:, 2:] = True
        assert torch.equal(got.isnan().all(2), want) and torch.equal(got.isnan().any(2), want)
        ref, tol = Step(seqs, 4, 2, 64, 16, dtype).reference()
        assert bool(((got.double() - ref).abs() <= tol)[~want].all())


# --------------------------------------- keys of very different sizes in a tile --
class Apart(Step):
    """Where contributions c = p scale lie far apart, the smallest step of float16, 2^-24, counts too.  Scales are taken as m
    over a power of two of their tile, 2^-5 (bfloat16, many rows: 2^-9) <= m < 1, or over their own, 1/2 <= m.  In float32
    weights are p m 2^x with x such that the largest p over that power has p 2^x = 2^14, so that the largest c has a weight of
    2^9 or more; each is off by 2^-25 at most, half the smallest step (of its second number too), which is 2^-34 of the largest
    c.  In bfloat16 weights are p 2^x with the largest 2^8 or more and meet values m v: 2^-25 m of at least 2^8 m', which is
    2^-33 m / m' <= 2^-24.  (Few rows are as float32.)  The output is off by that times the sum of the 8-bit values of the keys seen.  Where a scale is zero,
    which counts as 2^-60, 2^-85 and 2^-92 a key come to it (test_attention_tiny_values)."""

    def reference(self):
        out, tol = super().reference()
        least = 2.0 ** (-34 if self.dtype == torch.float32 else -24)
        for s, (n, x) in enumerate(self.seqs):
            lo, j = int(self.q_off[s]), torch.arange(x)
            page = self.pages[s].long()[j // self.page]
            k, _ = self.rows(s)
            seen = torch.stack([self.sees(s, i) for i in range(n)])
            for h in range(self.heads):
                c = h // (self.heads // self.kv)
                y = torch.where(seen, self.q[lo:lo + n, h].double() @ k[c].T * self.scale, -torch.inf)
                most = (torch.softmax(y, 1).nan_to_num(0.0) * self.vs[page, c, j % self.page].double()).amax(1, keepdim=True)
                v8 = self.v[page, c, j % self.page, :self.d].double().abs()
                zero = 2.0 ** -85 + x * 2.0 ** -92 if bool((self.vs[page, c, j % self.page] == 0).any()) else 0.0
                tol[lo:lo + n, h] += 1.05 * (least * most * (seen.double() @ v8) + zero)
        return out, tol

    def check_but(self, keys):
        """Rows that see none of the keys range(*keys[s]) of their sequence s, whose scores are too large for errors of the first
        order."""
        got, (ref, tol) = self.run(), self.reference()
        some = False
        for s, (n, x) in enumerate(self.seqs):
            for i in range(n):
                if not bool(self.sees(s, i)[keys[s][0]:keys[s][1]].any()):
                    r = int(self.q_off[s]) + i
                    assert bool(((got[r].double() - ref[r]).abs() <= tol[r]).all()), (s, i)
                    some = True
        assert some


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("which, factor", [("vs", 2.0 ** 40), ("vs", 2.0 ** -40), ("ks", 2.0 ** 30), ("vs", 2.0 ** 18), ("ks", 2.0 ** -30)])
def test_attention_keys_that_some_rows_do_not_see(which, factor, d, dtype):
    """The last keys are 2^40 times the others, or their fraction: queries before them are none the worse for it."""
    for seqs in ([(4, 100), (2, 64), (1, 30)], [(100, 150), (40, 40)], [(2, 5003)], [(60, 3001)]):
        step = Apart(seqs, 4, 2, d, 16, dtype)
        keys = [(x - max(1, n // 2), x) for n, x in seqs]
        for s, at in enumerate(keys):
            scale_keys(step, which, s, range(*at), factor)
        step.check() if factor < 2.0 ** 30 or which == "vs" else step.check_but(keys)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("which, factor", [("vs", 2.0 ** 40), ("ks", 2.0 ** 30)])
def test_attention_keys_that_leave_the_window(which, factor, dtype):
    """The first keys of a window are large: rows whose window begins behind them are none the worse for it."""
    for seqs in ([(4, 100), (2, 64)], [(100, 250), (40, 140)]):
        step = Apart(seqs, 4, 2, 64, 16, dtype, window=33, sinks=2)
        keys = [(x - n - 32, x - n - 32 + n // 2) for n, x in seqs]
        for s, at in enumerate(keys):
            scale_keys(step, which, s, range(*at), factor)
        step.check() if which == "vs" else step.check_but(keys)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("n", [6, 40])
def test_attention_other_branches_of_a_tree_may_be_large(n, dtype):
    tree = [m for _ in range(3) for m in branches(n, gen(n))]
    for which, factor in (("vs", 2.0 ** 40), ("ks", 2.0 ** 30)):
        step = Apart([(n, n), (n, n + 63), (n, n + 300)], 4, 2, 64, 16, dtype, tree=tree)
        keys = [(x - n // 2, x) for _, x in step.seqs]
        for s, at in enumerate(keys):
            scale_keys(step, which, s, range(*at), factor)
        step.check() if which == "vs" else step.check_but(keys)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 128, 200])
def test_attention_a_large_value_of_no_weight(d, dtype):
    """A key whose score lies far below the others' has a value 2^40 times theirs: it takes no bits from them."""
    for n in (1, 100):
        for at in (5, 130, n + 190):
            step = Apart([(n, n + 200)], 4, 2, d, 16, dtype)
            page = int(step.pages[0, at // 16])
            step.q[:] = step.q[:1]
            step.k[page, :, at % 16, :d] = (step.q[0, ::2].float() * -40).round().clamp(-127, 127).to(torch.int8)
            step.q[:, 1::2] = step.q[:, ::2]
            scale_keys(step, "ks", 0, [at], 8.0)
            scale_keys(step, "vs", 0, [at], 2.0 ** 40)
            step.check()


# -------------------------------------------------- queries of different sizes --
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 128, 200])
def test_attention_a_large_query_takes_no_bits_from_others(d, dtype):
    """One head of one token is 2^32 times the others, which lie in its row block."""
    for seqs in ([(4, 100), (1, 30)], [(8, 90), (1, 30)], [(100, 150), (40, 40)]):
        step = Step(seqs, 4, 2, d, 16, dtype)
        step.q[2, 1] = (step.q[2, 1].float() * 2.0 ** 32).to(dtype)
        got, (ref, tol) = step.run(), step.reference()
        keep = torch.ones(step.T, 4, dtype=torch.bool)
        keep[2, 1] = False
        assert bool(((got.double() - ref).abs() <= tol)[keep].all())


# ------------------------------------------------------------------ large scores --
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 128, 200])
def test_attention_large_scores(d, dtype):
    """Scores up to 2^45, of which one lies above all others by a third and more: the output is that key's value, off by its
    rounding and its weight's (2 h in bfloat16), float32 roundings and the output's own."""
    tol = 1.01 * ((2 * H if dtype == torch.bfloat16 else 2 * H * H) + 16 * V + half(dtype))
    for seqs in ([(1, 200), (3, 200)], [(60, 200)], [(1, 4000)], [(50, 3000)]):
        for size in range(8, 42, 3):
            step = Step(seqs, 4, 2, d, 16, dtype)
            step.q[:] = step.q[:1]
            step.q[:, 1::2] = step.q[:, ::2]
            step.ks[:] = 0.02 * 2.0 ** size
            at = 7 * size % 140
            for s in range(len(seqs)):
                page = int(step.pages[s, at // 16])
                step.k[page, :, at % 16, :d] = (step.q[0, ::2].float() * 40).round().clamp(-127, 127).to(torch.int8)
            got = step.run()
            for s, (n, x) in enumerate(seqs):
                lo = int(step.q_off[s])
                _, v = step.rows(s)
                want = v[:, at].repeat_interleave(2, 0)[None].expand(n, 4, d)
                ok = (got[lo:lo + n].double() - want).abs() <= tol * want.abs()
                assert bool(ok.all()), (seqs, s, size)


# ---------------------------------------------------------------- another plan --
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 256])
def test_attention_counts_a_call_on_another_plan_once(d, dtype):
    for n in (1, 100):
        a = Step([(n, 150 + 20 * i) for i in range(5)] + [(1, 700)], 4, 2, d, 16, dtype).load()
        b = Step([(n, 150 + 20 * i) for i in range(5)] + [(1, 700)], 4, 2, d, 16, dtype, window=2 ** 20).load()
        out = torch.full(a.q.shape, 7.0, dtype=dtype, device="cuda:0")
        plan = torch.zeros(max(a.plan.numel(), b.plan.numel()), dtype=torch.uint8, device="cuda:0")
        plan[:b.plan.numel()] = b.plan
        for calls in (1, 2, 3):
            L.lora_attention_apply(a.attention, a.cache, a.batch, plan, a.q.to("cuda:0"), out, a.ws)
            assert L.lora_read_device_errors(plan) == calls
        assert bool((out == 7).all())


# -------------------------------------------------------------------- tiny values --
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("size", [-58, -64, -72, -84, -96])
def test_attention_tiny_values(size, d, dtype):
    """Scales of values below 2^-60 lose bits: an output is off by 2^-85 more (values as float16 over 2^-60, whose smallest
    step is 2^-24) and by 2^-92 a key (weights over 2^-60, which are 2^14 at most)."""
    for seqs in ([(1, 300), (2, 90)], [(100, 150)], [(2, 5000)]):
        step = Step(seqs, 4, 2, d, 16, dtype)
        step.vs *= 2.0 ** size / 0.02
        got, (ref, tol) = step.run(), step.reference()
        for s, (n, x) in enumerate(seqs):
            lo = int(step.q_off[s])
            more = 1.05 * (2.0 ** -85 + x * 2.0 ** -92) if size < -59 else 0.0
            assert bool(((got[lo:lo + n].double() - ref[lo:lo + n]).abs() <= tol[lo:lo + n] + more).all())


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 128, 200])
def test_attention_a_zero_value_of_most_weight(d, dtype):
    """A key takes nearly all of the softmax and adds nothing: what the others add is small, and right all the same."""
    for n in (1, 100):
        for at in (5, 130):
            for factor in (1.0, 2.0):
                step = Apart([(n, n + 200)], 4, 2, d, 16, dtype)
                page = int(step.pages[0, at // 16])
                step.q[:] = step.q[:1]
                step.q[:, 1::2] = step.q[:, ::2]
                step.k[page, :, at % 16, :d] = (step.q[0, ::2].float() * 40).round().clamp(-127, 127).to(torch.int8)
                scale_keys(step, "ks", 0, [at], factor)
                scale_keys(step, "vs", 0, [at], 0.0)
                step.check()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("d", [64, 128, 200])
def test_attention_one_key_of_a_tile_of_many_sizes(d, dtype):
    """Each query sees its own key alone, among others of 2^-20 to 2^20 of its size: the output is that key's value, off by the
    roundings of its weight (h^2 in float32; in bfloat16 h, and h of the value), 8 float32 roundings and the output's own."""
    tol = 1.01 * ((2 * H if dtype == torch.bfloat16 else H * H) + 8 * V + half(dtype))
    for seqs in ([(3, 100), (2, 40), (1, 9)], [(100, 300), (40, 40)]):
        step = Step(seqs, 4, 2, d, 16, dtype, window=1)
        step.vs *= 2.0 ** torch.randint(-20, 21, step.vs.shape, generator=gen(d))
        got = step.run()
        for s, (n, x) in enumerate(seqs):
            lo = int(step.q_off[s])
            want = step.rows(s)[1][:, x - n:].repeat_interleave(2, 0).transpose(0, 1)
            assert bool(((got[lo:lo + n].double() - want).abs() <= tol * want.abs()).all()), (seqs, s)

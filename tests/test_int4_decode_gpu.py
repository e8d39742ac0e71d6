"""Attention over a 4-bit cache on the GPU, single tokens and verify steps,
against float64 attention over the dequantised cache.

Tolerance of an output (derived before the first run): the bf16 output is off
by at most 2^-8 of itself; P' = p * scale is rounded to f16, 2^-11 of itself,
so the sum by at most 2^-11 sum p|v|; a raw score is a sum of 128 products in
fp32 that starts at the codes' offset, off by at most 33 additions of 2^-23 of
a partial sum of at most 23 sum|q| scale in each group, which for the normal
queries and keys here (sum over a group |q| <= 45, scale <= 0.75, softmax scale
0.0884) is 33 2^-23 23 45 0.75 0.0884 4 = 1.1e-3 in the exponent at the very
most, on p and on the sum of p: 2.2e-3 sum p|v|.  Together 2^-8 |ref| + 2.7e-3 sum p|v|.
In the 2-norm the roundings are at most 2^-8 of the result."""
import numpy as np
import pytest
import torch

from paged_kv_flash_gb300 import workloads as W
from tests import int4_ref as R
from tests.helpers import check_lse, dev, dev_bf16, host_f32

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def pk():
    from paged_kv_flash_gb300 import pagedkv
    return pagedkv


def close(got, ref, mag, what=""):
    g = host_f32(got).astype(np.float64)
    assert g.shape == ref.shape and np.isfinite(g).all(), what
    err = np.abs(g - ref)
    bad = err > 2.0 ** -8 * np.abs(ref) + 2.7e-3 * mag
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, max {err.max():.3e}"
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(g - ref) <= 2.0 ** -8 * norm, f"{what}: 2-norm"


class Case:
    def __init__(self, seed, lens, Hq, Hkv, counts=None, smooth=False):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        self.layout = W.scatter_pages(rng, self.lens)
        self.w = W.smoothing_weight(rng) if smooth else None
        self.k, self.v = R.fill(rng, self.layout, self.lens, Hkv, self.w)
        self.counts = np.ones(len(lens), np.int64) if counts is None else np.asarray(counts)
        self.cu = W.cu_from_counts(self.counts)
        self.q = W.normal_bf16(rng, (int(self.counts.sum()), Hq, 128))

    def ref(self, scale=SCALE):
        return R.attention(self.k, self.v, W.bits_to_float(self.q).astype(np.float64), self.cu,
                           self.layout.block_table, self.lens, scale, self.w)

    def args(self, pk):
        pool = pk.Pool(dev(self.k), dev(self.v))
        return (pool, dev_bf16(self.q), dev(self.layout.block_table), dev(self.lens),
                int(self.lens.max()))

    def smooth(self):
        return None if self.w is None else dev(self.w)

    def decode(self, pk, splits=0, scale=SCALE, fn="paged_attn_decode", **kw):
        out, lse = getattr(pk, fn)(*self.args(pk), scale, k_smooth=self.smooth(),
                                   num_splits=splits, **kw)
        assert pk.poll_device_error() == pk.OK
        return out, lse

    def multi(self, pk, splits=0, max_q=None, poll=True):
        pool, q, bt, lens, ml = self.args(pk)
        out, lse = pk.paged_attn_decode_multi(
            pool, q, dev(self.cu), bt, lens, int(self.counts.max()) if max_q is None else max_q,
            ml, SCALE, num_splits=splits, k_smooth=self.smooth())
        if poll:
            assert pk.poll_device_error() == pk.OK
        return out, lse


# ------------------------------------------------------------ single tokens

@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 8, 9, 20, 40])
def test_decode_ragged_lengths_and_group_sizes(pk, G, smooth):
    """Lengths 0, 1, around a page, a tile of pages and several splits; every
    slot past a length is poisoned (NaN scales)."""
    c = Case(2000 + G, [0, 1, 15, 16, 17, 63, 64, 65, 777, 1500], 2 * G, 2, smooth=smooth)
    ro, rl, mag = c.ref()
    for splits in (0, 1, 3, 7):
        out, lse = c.decode(pk, splits)
        close(out, ro, mag, what=f"G={G} splits={splits}")
        check_lse(lse, rl, f"G={G} splits={splits}")
        assert (host_f32(out)[0] == 0).all() and np.isneginf(lse[0].cpu().numpy()).all()


@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_decode_kv_heads(pk, Hkv):
    c = Case(2100 + Hkv, [300, 45], 4 * Hkv, Hkv)
    ro, rl, mag = c.ref()
    out, lse = c.decode(pk)
    close(out, ro, mag)
    check_lse(lse, rl)


def test_decode_long_sequence(pk):
    c = Case(2110, [32768], 8, 2, smooth=True)
    ro, rl, mag = c.ref()
    for splits in (0, 2):
        out, lse = c.decode(pk, splits)
        g = host_f32(out).astype(np.float64)
        # outputs are ~ sqrt(128) ... small against v; the 2-norm bar is the sharp one
        assert np.linalg.norm(g - ro) <= 2.0 ** -8 * np.linalg.norm(ro)
        check_lse(lse, rl)


def test_fused_merge_and_noalloc_are_bit_identical(pk):
    """The three forms of the call, and a workspace reused by calls of other
    shapes, row groups among them (20 query heads per KV head: one CTA; 40: two)."""
    ws = pk.decode_workspace(1 << 24, 1 << 18)
    for G, lens in ((4, [700, 40, 0, 1023]), (40, [300, 700]), (3, [2000]), (4, [16, 5])):
        c = Case(2120 + G, lens, 2 * G, 2)
        for splits in (0, 5):
            a = c.decode(pk, splits, workspace=ws)
            f = c.decode(pk, splits, workspace=ws, fused=True)
            n = c.decode(pk, splits, fn="paged_attn_decode_noalloc")
            for x in (f, n):
                assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])
            assert (ws[:1 << 18] == 0).all()                 # the counters are zero again
        ro, _, mag = c.ref()
        close(a[0], ro, mag)


def test_decode_without_lse_and_into_given_buffers(pk):
    c = Case(2130, [130], 8, 2)
    out = torch.full((1, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = c.decode(pk, out=out, want_lse=False)
    assert o.data_ptr() == out.data_ptr() and lse is None
    ro, _, mag = c.ref()
    close(out, ro, mag)


@pytest.mark.parametrize("k", [-40, -20, 20, 40])
def test_query_magnitude_is_exact(pk, k):
    """q 2^k with the softmax scale 2^-k: the same bits (powers of two leave
    every step but the query's own normalisation as it was)."""
    c = Case(2140, [500, 33], 8, 2)
    a = c.decode(pk, 3)
    c.q = W.to_bf16_bits(W.bits_to_float(c.q) * np.float32(2.0 ** k))
    b = c.decode(pk, 3, scale=SCALE * 2.0 ** -k)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def scales_of(pool):
    return pool[..., 1024:].view(np.float16)


@pytest.mark.parametrize("factor", [2.0 ** -12, 2.0 ** -6, 2.0 ** 8, 2.0 ** 15])
def test_value_magnitude(pk, factor):
    """V scales from subnormal fp16 to the largest: outputs scale with them."""
    c = Case(2150, [600, 21], 8, 2, smooth=True)
    s = scales_of(c.v)
    with np.errstate(over="ignore", invalid="ignore"):
        s[...] = np.minimum(s.astype(np.float64) * factor, 65504).astype(np.float16)
    ro, rl, mag = c.ref()
    out, lse = c.decode(pk)
    close(out, ro, mag)
    check_lse(lse, rl)


def test_value_magnitudes_that_differ_between_keys(pk):
    """Keys of large V and small score beside keys of small V and large score,
    in either order, all-zero V first: P' stays in f16's range."""
    for order in (1, -1):
        c = Case(2160, [16 * 64], 4, 1)
        pages = c.layout.block_table[0][::order]
        f = 2.0 ** np.linspace(-13, 15, 64)
        for i, p in enumerate(pages):
            s = scales_of(c.v[p:p + 1])
            s[...] = np.minimum(s.astype(np.float64) * f[i], 65504).astype(np.float16) if i % 7 else 0
        ro, rl, mag = c.ref()
        for splits in (1, 4):
            out, lse = c.decode(pk, splits)
            close(out, ro, mag)
            check_lse(lse, rl)


def test_extreme_scores_one_key_takes_all(pk):
    """Scores far apart: one key has all the weight, and lse follows it."""
    c = Case(2170, [200, 200], 8, 2)
    _, rl, _ = c.ref(scale=30.0)
    out, lse = c.decode(pk, 3, scale=30.0)
    g = host_f32(out).astype(np.float64)
    # scores of ~ 30 * 11 * 3: the fp32 bound above grows by 30 / 0.0884; compare where it decides
    # nothing: rows whose two largest scores are more than 2 apart
    assert np.isfinite(g).all()
    assert np.abs(lse.cpu().numpy() - rl).max() <= 1.1e-3 * 30 / SCALE + 1e-3
    for scale in (0.0, -SCALE):
        ro, rl, mag = c.ref(scale=scale)
        out, lse = c.decode(pk, 3, scale=scale)
        close(out, ro, mag, what=f"scale {scale}")
        check_lse(lse, rl)


def test_nan_groups_reach_only_their_rows(pk):
    """A NaN scale, in K or in V, makes the rows of its KV head NaN (of V: its
    group's channels at least); other heads and sequences keep their bits."""
    for which in ("v", "k"):
        c = Case(2180, [100, 100], 8, 2)
        clean = host_f32(c.decode(pk)[0])
        page, slot = c.layout.block_table[0, 3], 5
        scales_of(getattr(c, which))[page, 1].reshape(16, 4)[slot, 2] = np.nan
        out = host_f32(c.decode(pk)[0])
        assert np.isnan(out[0, 4:, 64:96]).all()
        assert which == "v" or np.isnan(out[0, 4:]).all()
        assert np.array_equal(out[0, :4], clean[0, :4]) and np.array_equal(out[1], clean[1])


def test_bad_pages_and_lengths_are_flagged(pk):
    c = Case(2190, [100, 40], 8, 2)
    pool, q, bt, lens, ml = c.args(pk)
    ro, _, mag = c.ref()
    for what in ("page", "negative", "length"):
        b2, l2 = bt.clone(), lens.clone()
        if what == "page":
            b2[1, 0] = pool.num_pages
        elif what == "negative":
            b2[1, 1] = -3
        else:
            l2[1] = bt.shape[1] * 16 + 1
        out, _ = pk.paged_attn_decode(pool, q, b2, l2, ml, SCALE)
        assert pk.poll_device_error() == pk.ERR_INVALID
        assert pk.poll_device_error() == pk.OK
        close(out[:1], ro[:1], mag[:1], what=what)                  # the other sequence is right


def test_captured_decode_follows_its_inputs(pk):
    """A captured decode replayed while another graph with its own workspace
    runs: outputs follow the lengths and queries written between replays."""
    c1, c2 = Case(2200, [400, 30], 8, 2), Case(2201, [350, 900], 8, 2)
    graphs, held = [], []                       # a graph keeps the addresses, not the tensors
    for c in (c1, c2):
        pool, q, bt, lens, ml = c.args(pk)
        _, _, nb, zb = pk.decode_plan(2, 8, 2, ml, 4, pk.INT4)
        ws = pk.decode_workspace(nb, zb)
        out, lse = torch.empty_like(q), torch.empty(2, 8, device="cuda")
        run = lambda: pk.paged_attn_decode(pool, q, bt, lens, ml, SCALE, num_splits=4,  # noqa: E731,B023
                                           workspace=ws, out=out, lse=lse)              # noqa: B023
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run()
        graphs.append((g, s, q, lens, out, lse))
        held.append((pool, bt, ws))
    for shrink in (0, 100, 399):
        for c, (g, s, q, lens, out, lse) in zip((c1, c2), graphs):
            c.lens = np.maximum(c.lens - shrink, 0).astype(np.int32)
            lens.copy_(dev(c.lens))
        torch.cuda.synchronize()
        for g, s, *_ in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert pk.poll_device_error() == pk.OK
        for c, (g, s, q, lens, out, lse) in zip((c1, c2), graphs):
            ro, rl, mag = c.ref()
            close(out, ro, mag, what=f"shrink {shrink}") if np.linalg.norm(ro) else None
            check_lse(lse, rl)


def test_pool_offsets_past_31_bits(pk):
    """A pool of more than 2^31 bytes: append, decode and unpack at its end."""
    Hkv, n = 8, 240000                                       # 240,000 x 8 x 1,152 = 2.2e9 bytes
    pool = pk.Pool.empty(n, Hkv, dtype=torch.uint8)
    rng = np.random.default_rng(2210)
    L = 40
    bt = np.array([[n - 1, n - 3, n - 2]], np.int32)
    kn, vn, q = (W.normal_bf16(rng, s) for s in ((L, Hkv, 128), (L, Hkv, 128), (1, Hkv, 128)))
    lens = dev(np.array([L], np.int32))
    pk.kv_append(pool, dev_bf16(kn), dev_bf16(vn), dev(W.cu_from_counts([L])), dev(bt), lens)
    out, lse = pk.paged_attn_decode(pool, dev_bf16(q), dev(bt), lens, L, SCALE)
    wide = pk.Pool.empty(3, Hkv)
    pk.kv_unpack(pool, wide, dev(bt), dev(np.array([[0, 1, 2]], np.int32)), lens, L)
    assert pk.poll_device_error() == pk.OK
    k, v = (t[n - 3:].cpu().numpy() for t in (pool.k, pool.v))
    local = np.array([[2, 0, 1]], np.int32)
    ro, rl, mag = R.attention(k, v, W.bits_to_float(q).astype(np.float64), [0, 1], local, [L], SCALE)
    close(out, ro, mag)
    check_lse(lse, rl)
    val = R.values(v[local[0]]).transpose(0, 2, 1, 3).reshape(-1, Hkv, 128)[:L]
    got = host_f32(wide.v).transpose(0, 2, 1, 3).reshape(-1, Hkv, 128)[:L]
    assert (np.abs(got - val) <= 2.0 ** -8 * np.abs(val)).all()


# --------------------------------------------------------------- verify steps

@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 8])
def test_verify_steps(pk, G, smooth):
    """Steps of 1, 2, 5, 16, 9 and no tokens; 16 tokens that are the whole
    sequence; contexts up to several splits, page borders inside a step."""
    c = Case(2300 + G, [40, 1024, 17, 777, 16, 300, 1], 2 * G, 2, counts=[1, 2, 5, 9, 16, 0, 1],
             smooth=smooth)
    ro, rl, mag = c.ref()
    for splits in (0, 1, 3, 7):
        out, lse = c.multi(pk, splits)
        close(out, ro, mag, what=f"G={G} splits={splits}")
        check_lse(lse, rl, f"G={G} splits={splits}")


@pytest.mark.parametrize("tokens", [1, 2, 4, 6, 8, 11, 16])
def test_verify_step_sizes(pk, tokens):
    """Every number of n-tiles and row groups of the kernel, odd ones among them."""
    for G in (1, 4, 5):
        c = Case(2400 + 10 * tokens + G, [200, 16 * 37], G, 1, counts=[tokens, tokens])
        ro, rl, mag = c.ref()
        out, lse = c.multi(pk)
        close(out, ro, mag, what=f"G={G}")
        check_lse(lse, rl)


def test_one_token_steps_are_decode(pk):
    c = Case(2500, [1, 300, 1025], 8, 2)
    a, b = c.decode(pk, 4), c.multi(pk, 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_step_longer_than_max_q_or_its_sequence_is_flagged(pk):
    c = Case(2510, [100, 200], 8, 2, counts=[3, 5])
    ro, _, mag = c.ref()
    out, _ = c.multi(pk, max_q=4, poll=False)
    assert pk.poll_device_error() == pk.ERR_INVALID
    close(out[:3], ro[:3], mag[:3])
    c.lens = np.array([2, 200], np.int32)                    # 3 tokens, 2 positions
    c.multi(pk, poll=False)
    assert pk.poll_device_error() == pk.ERR_INVALID
    assert pk.poll_device_error() == pk.OK


@pytest.mark.parametrize("splits", [1, 3, 12])
@pytest.mark.parametrize("G", [2, 8])
def test_positions_a_row_does_not_see_may_hold_nan(pk, G, splits):
    """NaN keys and values of the step's last two tokens reach the rows that see
    them, and no earlier row."""
    c = Case(2530 + G, [200, 77], 2 * G, 2, counts=[4, 5])
    ro, rl, mag = c.ref()
    for b in range(2):
        for p in (c.lens[b] - 2, c.lens[b] - 1):
            page = c.layout.block_table[b, p // 16]
            for pool in (c.k, c.v):
                scales_of(pool)[page].reshape(2, 16, 4)[:, p % 16] = np.nan
    out, lse = c.multi(pk, splits)
    early = [0, 1, 4, 5, 6]
    close(out[early], ro[early], mag[early])
    check_lse(lse[early], rl[early])
    assert torch.isnan(out[[2, 3, 7, 8]]).all()


@pytest.mark.parametrize("many", [False, True])
def test_padded_and_skipped_rows_are_left_as_they_were(pk, many):
    """Rows behind the last sequence, of a sequence without tokens and of a
    skipped one; splits merged in clusters (few) and by the combine (many)."""
    B = 80 if many else 3
    counts = np.where(np.arange(B) % 3 == 1, 6, 3)
    c = Case(2540, np.full(B, 300), 8, 2, counts=counts)
    pool, _, bt, lens, ml = c.args(pk)
    T = int(c.cu[-1])
    q = torch.zeros((T + 7, 8, 128), dtype=torch.bfloat16, device="cuda")
    q[:T] = dev_bf16(c.q)
    out = torch.full_like(q, 7.0)
    lse = torch.full((T + 7, 8), 7.0, device="cuda")
    pk.paged_attn_decode_multi(pool, q, dev(c.cu), bt, lens, 5, ml, SCALE, num_splits=8, out=out,
                               lse=lse)
    assert pk.poll_device_error() == pk.ERR_INVALID          # six tokens of at most five
    skipped = torch.ones(T + 7, dtype=torch.bool)
    for b in np.nonzero(counts <= 5)[0]:
        skipped[c.cu[b]:c.cu[b + 1]] = False
    assert (out[skipped.cuda()] == 7).all() and (lse[skipped.cuda()] == 7).all()
    rows = np.nonzero(~skipped.numpy())[0][:30]
    ro, rl, mag = c.ref()
    close(out[torch.from_numpy(rows).cuda()], ro[rows], mag[rows])


def test_bf16_padded_rows_are_left_as_they_were(pk):
    rng = np.random.default_rng(2545)
    lens = np.array([300, 200], np.int32)
    layout = W.scatter_pages(rng, lens)
    pool = pk.Pool(*(dev_bf16(W.normal_bf16(rng, (layout.num_pages, 2, 16, 128)))
                     for _ in range(2)))
    q = dev_bf16(W.normal_bf16(rng, (12, 8, 128)))
    out = torch.full_like(q, 7.0)
    args = (dev(W.cu_from_counts([3, 4])), dev(layout.block_table), dev(lens), 4, 300, SCALE)
    pk.paged_attn_decode_multi(pool, q, *args, num_splits=4, out=out)
    want, _ = pk.paged_attn_decode_multi(pool, q[:7].contiguous(), *args, num_splits=4)
    assert pk.poll_device_error() == pk.OK
    assert torch.equal(out[:7], want) and (out[7:] == 7).all()


@pytest.mark.parametrize("splits", [1, 2, 8, 20])
def test_lengths_past_the_plan_are_flagged(pk, splits):
    """max_seq_len below a length that the block table still holds: an error, the
    other sequences right, the next (fused) call right."""
    c = Case(2550, [640, 320, 100], 8, 2)
    pool, q, bt, lens, _ = c.args(pk)
    ro, _, mag = c.ref()
    _, _, wsb, zero = pk.decode_plan(3, 8, 2, 640, splits, pk.INT4)
    ws = torch.zeros(max(wsb, 256), dtype=torch.uint8, device="cuda")
    for fused in (False, True):
        out, _ = pk.paged_attn_decode(pool, q, bt, lens, 320, SCALE, num_splits=splits,
                                      workspace=ws, fused=fused)
        assert pk.poll_device_error() == pk.ERR_INVALID
        close(out[1:], ro[1:], mag[1:])
        assert torch.isfinite(out).all()
        out, _ = pk.paged_attn_decode(pool, q, bt, lens, 640, SCALE, num_splits=splits,
                                      workspace=ws, fused=fused)
        assert pk.poll_device_error() == pk.OK
        close(out, ro, mag)
    cu = dev(W.cu_from_counts([1, 1, 1]))
    out, _ = pk.paged_attn_decode_multi(pool, q, cu, bt, lens, 1, 320, SCALE, num_splits=splits)
    assert pk.poll_device_error() == pk.ERR_INVALID
    close(out[1:], ro[1:], mag[1:])


def test_append_decode_verify_run_together(pk):
    """A request's life on a 4-bit cache with smoothed keys: tables, append of
    the prompt, a verify step, then single tokens; each against float64."""
    rng = np.random.default_rng(2520)
    B, Hq, Hkv = 3, 8, 2
    w = W.smoothing_weight(rng)
    pool = pk.Pool.empty(64, Hkv, dtype=torch.uint8)
    bt = torch.full((B, 16), -1, dtype=torch.int32, device="cuda")
    ring = dev(rng.permutation(64).astype(np.int32))
    state = dev(np.array([5, 59], np.int32))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    for new in ([30, 100, 7], [4, 1, 16], [1, 1, 1], [0, 1, 0]):
        T = sum(new)
        cu, _ = pk.page_tables(lens, dev(np.array(new, np.int32)), bt, ring, state, 64)
        kn = W.keys_with_channel_weight(rng, (T, Hkv, 128), w)
        vn, q = W.normal_bf16(rng, (T, Hkv, 128)), W.normal_bf16(rng, (T, Hq, 128))
        pk.kv_append(pool, dev_bf16(kn), dev_bf16(vn), cu, bt, lens, k_smooth=dev(w))
        if max(new) <= 16:
            out, lse = pk.paged_attn_decode_multi(pool, dev_bf16(q), cu, bt, lens, max(new), 256,
                                                  SCALE, k_smooth=dev(w))
            ro, rl, mag = R.attention(pool.k.cpu().numpy(), pool.v.cpu().numpy(),
                                 W.bits_to_float(q).astype(np.float64), cu.cpu().numpy(),
                                 bt.cpu().numpy(), lens.cpu().numpy(), SCALE, w)
            close(out, ro, mag, what=str(new))
            check_lse(lse, rl, str(new))
        assert pk.poll_device_error() == pk.OK


# ------------------------------------------------- more than one wave of CTAs

def long_batch(seed, B, lens_of, Hq, Hkv, counts=None, smooth=False):
    """More work than one wave of CTAs: B sequences whose cached positions share
    a few pages of random data (the block tables repeat them), so that the
    float64 reference stays small."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens_of(rng, B), np.int32)
    c = Case(seed, [16 * 24], Hq, Hkv, counts=[1], smooth=smooth)
    table = rng.choice(c.layout.block_table[0], (B, -(-int(lens.max()) // 16))).astype(np.int32)
    c.layout = W.Layout(c.layout.num_pages, table, c.layout.sentinel_page)
    c.lens = lens
    c.counts = np.ones(B, np.int64) if counts is None else np.asarray(counts)
    c.cu = W.cu_from_counts(c.counts)
    c.q = W.normal_bf16(rng, (int(c.counts.sum()), Hq, 128))
    return c


def sampled_ref(c, rows):
    """The reference of some rows (token t of sequence b alone)."""
    out, lse, mag = [], [], []
    for t in rows:
        b = int(np.searchsorted(c.cu, t, side="right")) - 1
        n = int(c.lens[b] - c.counts[b] + (t - c.cu[b]) + 1)
        o = R.attention(c.k, c.v, W.bits_to_float(c.q[t:t + 1]).astype(np.float64), [0, 1],
                        c.layout.block_table[b:b + 1], [n], SCALE, c.w)
        for acc, x in zip((out, lse, mag), o):
            acc.append(x[0])
    return np.stack(out), np.stack(lse), np.stack(mag)


LENGTHS = {
    "ragged": lambda rng, B: rng.integers(0, 4200, B),
    "one long": lambda rng, B: np.where(np.arange(B) == B // 2, 20000, rng.integers(0, 40, B)),
    "zeros between": lambda rng, B: np.where(np.arange(B) % 3 == 1, 3000, 0),
    "equal": lambda rng, B: np.full(B, 3333),
}


@pytest.mark.parametrize("G,smooth", [(4, False), (4, True), (8, False), (12, True)])
@pytest.mark.parametrize("kind", sorted(LENGTHS))
def test_large_batches(pk, kind, G, smooth):
    B, Hkv = 90, 8
    c = long_batch(2600 + G, B, LENGTHS[kind], G * Hkv, Hkv, smooth=smooth)
    out, lse = c.decode(pk)
    rows = np.unique(np.concatenate([np.random.default_rng(7).integers(0, B, 10),
                                     np.flatnonzero(c.lens == 0)[:2], [c.lens.argmax(), B - 1]]))
    ro, rl, mag = sampled_ref(c, rows)
    idx = torch.from_numpy(rows).cuda()
    close(out[idx], ro, mag, what=kind)
    check_lse(lse[idx], rl, kind)
    # every row, the sampled ones or not, as other splits give it
    fo, fl = c.decode(pk, fused=True)
    assert torch.equal(out, fo) and torch.equal(lse, fl)
    # (the call without workspace takes fewer splits where its 16 MiB are short)
    for go, gl in (c.decode(pk, 3), c.decode(pk, fn="paged_attn_decode_noalloc")):
        d = (out.float() - go.float()).abs()
        assert (d <= 2.0 ** -7 * go.float().abs() + 2 * 2.7e-3 * 6).all()
        same = torch.isneginf(lse) & torch.isneginf(gl)
        assert ((lse - gl).abs().masked_fill(same, 0) <= 2e-3).all()


@pytest.mark.parametrize("smooth", [False, True])
def test_large_batches_of_verify_steps(pk, smooth):
    """Ragged steps (none, one, many tokens; one to eight row groups) and lengths."""
    rng = np.random.default_rng(2700)
    B, Hkv, G = 30, 8, 4
    counts = rng.integers(0, 17, B)
    counts[:3] = [0, 16, 1]
    c = long_batch(2701, B, lambda r, n: np.maximum(r.integers(1, 4000, n), counts), G * Hkv, Hkv,
                   counts=counts, smooth=smooth)
    out, lse = c.multi(pk, max_q=16)
    rows = np.unique(np.concatenate([c.cu[:-1][counts > 0][:8], c.cu[1:][counts > 0][:8] - 1]))
    ro, rl, mag = sampled_ref(c, rows)
    idx = torch.from_numpy(rows.astype(np.int64)).cuda()
    close(out[idx], ro, mag)
    check_lse(lse[idx], rl)
    go, gl = c.multi(pk, 3, max_q=16)
    assert ((out.float() - go.float()).abs() <= 2.0 ** -7 * go.float().abs() + 2 * 2.7e-3 * 6).all()
    assert ((lse - gl).abs() <= 2e-3).all()


def test_bad_sequences_in_a_large_batch_leave_the_rest_right(pk):
    c = long_batch(2800, 90, LENGTHS["ragged"], 32, 8)
    c.lens[:] = np.maximum(c.lens, 1)
    good, _ = c.decode(pk)
    pool, q, bt, lens, ml = c.args(pk)
    lens[5], bt[7, 0] = -1, pool.num_pages
    lens[6] = bt.shape[1] * 16 + 1
    out, lse = pk.paged_attn_decode(pool, q, bt, lens, ml, SCALE)
    assert pk.poll_device_error() == pk.ERR_INVALID
    assert pk.poll_device_error() == pk.OK
    keep = torch.ones(90, dtype=torch.bool, device="cuda")
    keep[5:8] = False
    d = (out.float() - good.float()).abs()[keep]
    assert (d <= 2.0 ** -7 * good.float().abs()[keep] + 2 * 2.7e-3 * 6).all()
    assert (out[5:7] == 0).all() and torch.isneginf(lse[5:7]).all()

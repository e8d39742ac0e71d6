"""The 4-bit cache's append and the unpacking of quantised pools on the GPU:
slabs, scales and bf16 pages bit for bit against the same IEEE fp32 steps in
numpy, and against the definition in float64."""
import numpy as np
import pytest
import torch

from paged_kv_flash_gb300 import workloads as W
from tests import int4_ref as R
from tests.helpers import dev, dev_bf16, host_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    from paged_kv_flash_gb300 import pagedkv
    return pagedkv


def empty(layout, Hkv, byte=0xA5):
    return np.full((layout.num_pages, Hkv, R.SLAB), byte, np.uint8)


def reference_append(k_pool, v_pool, kn, vn, cu, layout, lens, w=None):
    k_pool, v_pool = k_pool.copy(), v_pool.copy()
    kf, vf = W.bits_to_float(kn).astype(np.float32), W.bits_to_float(vn).astype(np.float32)
    if w is not None:
        kf = kf / w
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            p = lens[b] - n + i
            for h in range(kn.shape[1]):
                for pool, x in ((k_pool, kf), (v_pool, vf)):
                    R.put(pool, layout.block_table[b, p // 16], h, p % 16,
                          *R.quantize(x[cu[b] + i, h]))
    return k_pool, v_pool


def run_append(pk, k0, v0, kn, vn, cu, layout, lens, w=None):
    pool = pk.Pool(dev(k0), dev(v0))
    pk.kv_append(pool, dev_bf16(kn), dev_bf16(vn), dev(cu), dev(layout.block_table),
                 dev(np.asarray(lens, np.int32)), k_smooth=None if w is None else dev(w))
    assert pk.poll_device_error() == pk.OK
    return pool.k.cpu().numpy(), pool.v.cpu().numpy()


@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("smooth", [False, True])
def test_append_is_bit_exact_and_touches_only_its_slots(pk, Hkv, smooth):
    """Ragged appends (one token, none, a page boundary, several pages), an odd
    head count; every other byte of the pool stays as it was."""
    rng = np.random.default_rng(900 + Hkv)
    counts, lens = np.array([1, 0, 20, 37]), np.array([16, 5, 33, 37], np.int32)
    layout = W.scatter_pages(rng, lens)
    cu = W.cu_from_counts(counts)
    w = W.smoothing_weight(rng) if smooth else None
    kn = W.normal_bf16(rng, (int(counts.sum()), Hkv, 128))
    vn = W.normal_bf16(rng, kn.shape)
    k0, v0 = empty(layout, Hkv), empty(layout, Hkv, 0x3C)
    want = reference_append(k0, v0, kn, vn, cu, layout, lens, w)
    got = run_append(pk, k0, v0, kn, vn, cu, layout, lens, w)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_append_error_is_at_most_half_a_step(pk):
    """In float64: |x - code * scale| <= scale / 2, plus 7 scale 2^-11 where the
    scale was rounded down below max|x| / 7 and the largest code saturates."""
    rng = np.random.default_rng(910)
    lens = np.array([64], np.int32)
    layout = W.scatter_pages(rng, lens)
    x = W.normal_bf16(rng, (64, 2, 128))
    k, v = run_append(pk, empty(layout, 2), empty(layout, 2), x, x, W.cu_from_counts([64]), layout,
                      lens)
    pages = layout.block_table[0, :4]
    for pool in (k, v):
        val = R.values(pool[pages]).transpose(0, 2, 1, 3).reshape(64, 2, 128)
        s = np.ascontiguousarray(pool[pages][..., 1024:]).view(np.float16).astype(np.float64)
        s = s.reshape(4, 2, 16, 4).transpose(0, 2, 1, 3).reshape(64, 2, 4).repeat(32, -1)
        err = np.abs(val - W.bits_to_float(x))
        assert (err <= s * (0.5 + 7 * 2.0 ** -11)).all()


def test_append_special_values(pk):
    """Zero groups, magnitudes whose scale is subnormal or rounds to zero,
    saturating magnitudes, and groups that hold a NaN or an infinity (NaN
    scale, codes 0) beside groups that do not."""
    rng = np.random.default_rng(911)
    x = rng.standard_normal((8, 1, 128)).astype(np.float32)
    x[0] = 0
    x[1, :, :32] = 0
    x[2] *= 1e-6                                     # subnormal fp16 scales
    x[3] *= 1e-9                                     # scales round to zero
    x[4] *= 1e6                                      # past 458,528: saturates
    x[5, 0, 40] = np.inf
    x[6, 0, 127] = np.nan
    x[7, 0, 0] = 3.0e38
    bits = W.to_bf16_bits(x)
    lens = np.array([8], np.int32)
    layout = W.scatter_pages(rng, lens)
    cu = W.cu_from_counts([8])
    k0 = empty(layout, 1)
    want = reference_append(k0, k0, bits, bits, cu, layout, lens)
    got = run_append(pk, k0, k0, bits, bits, cu, layout, lens)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    val = R.values(got[0][layout.block_table[0, :1]])[0, 0]
    assert (val[0] == 0).all() and (val[3] == 0).all()
    assert np.abs(val[4]).max() <= 7 * 65504.0
    assert np.isnan(val[5, 32:64]).all() and np.isfinite(val[5, :32]).all()
    assert np.isnan(val[6, 96:]).all() and np.isfinite(val[6, :96]).all()


def test_append_bad_page_is_flagged_and_skipped(pk):
    rng = np.random.default_rng(912)
    lens = np.array([16, 16], np.int32)
    layout = W.scatter_pages(rng, lens)
    layout.block_table[1, 0] = layout.num_pages          # outside the pool
    kn = W.normal_bf16(rng, (2, 2, 128))
    pool = pk.Pool(dev(empty(layout, 2)), dev(empty(layout, 2)))
    pk.kv_append(pool, dev_bf16(kn), dev_bf16(kn), dev(W.cu_from_counts([1, 1])),
                 dev(layout.block_table), dev(lens))
    assert pk.poll_device_error() == pk.ERR_INVALID
    want, _ = reference_append(empty(layout, 2), empty(layout, 2), kn[:1], kn[:1],
                               W.cu_from_counts([1]), layout, lens[:1])
    assert np.array_equal(pool.k.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8, torch.uint8])
@pytest.mark.parametrize("counts", [[2, 0, 3], [0, 0, 0]])
def test_rows_behind_the_last_sequence_are_left_out(pk, dtype, counts):
    """A padded batch: the pool is the one that the rows of the sequences alone
    leave, although the last one's table goes on."""
    rng = np.random.default_rng(913)
    lens = np.array([20, 7, 33], np.int32)
    layout = W.scatter_pages(rng, lens + 16)
    total = sum(counts)
    kn = dev_bf16(W.normal_bf16(rng, (total + 9, 2, 128)))
    pools = []
    for n in (total, total + 9):
        pool = pk.Pool.empty(layout.num_pages, 2, dtype=dtype)
        for t in (pool.k, pool.v, pool.k_scale, pool.v_scale):
            if t is not None:
                t.zero_()
        pk.kv_append(pool, kn[:n], kn[:n], dev(W.cu_from_counts(counts)),
                     dev(layout.block_table), dev(lens))
        assert pk.poll_device_error() == pk.OK
        pools.append(pool)
    for a, b in zip(*((p.k, p.v, p.k_scale, p.v_scale) for p in pools)):
        assert a is None or torch.equal(a, b)
    assert total == 0 or pools[1].k.float().abs().sum() > 0


def test_fused_inputs_leave_out_rows_behind_the_last_sequence(pk):
    rng = np.random.default_rng(914)
    lens, counts = np.array([20, 7], np.int32), [2, 1]
    layout = W.scatter_pages(rng, lens + 16)
    qkv = dev_bf16(W.normal_bf16(rng, (8, 4 + 2 * 2, 128)))
    pools, outs = [], []
    for n in (3, 8):
        pool = pk.Pool.empty(layout.num_pages, 2)
        pool.k.zero_(), pool.v.zero_()
        out = torch.full((n, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        pk.qkv_norm_rope_append(pool, qkv[:n], 4, dev(W.cu_from_counts(counts)),
                                dev(layout.block_table), dev(lens), q_out=out)
        assert pk.poll_device_error() == pk.OK
        pools.append(pool)
        outs.append(out)
    assert torch.equal(pools[0].k, pools[1].k) and torch.equal(pools[0].v, pools[1].v)
    assert torch.equal(outs[0], outs[1][:3]) and (outs[1][3:] == 5).all()


# ------------------------------------------------------------------- unpack

def wide_layout(rng, lens, starts):
    """A small staging pool: pages only for the logical pages that hold a
    position of the range; other entries name a page that does not exist."""
    width = max(1, int(-(-np.max(lens) // 16)))
    bt = np.full((len(lens), width), -7, np.int32)
    n = 0
    for b, (s, e) in enumerate(zip(starts, lens)):
        for lp in range(s // 16, -(-e // 16) if e > s else s // 16):
            bt[b, lp] = n
            n += 1
    perm = rng.permutation(max(n, 1)).astype(np.int32)
    return np.where(bt >= 0, perm[np.maximum(bt, 0)], bt).astype(np.int32), max(n, 1)


def expected_unpack(vals, w, bt, wide_bt, lens, starts, pages, fill):
    """bf16 bits of fp32(fp32(code * scale) * w); vals = fp32 code * scale."""
    out = np.full((pages, vals.shape[1], 16, 128), fill, np.uint16)
    for b in range(len(lens)):
        for p in range(starts[b], lens[b]):
            x = vals[bt[b, p // 16], :, p % 16]
            x = x * w if w is not None else x
            out[wide_bt[b, p // 16], :, p % 16] = W.to_bf16_bits(x)
    return out


@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_unpack_is_bit_exact_and_touches_only_its_range(pk, bits, smooth, Hkv):
    rng = np.random.default_rng(920 + Hkv)
    lens = np.array([1, 0, 16, 47, 130], np.int32)
    starts = np.array([0, 0, 3, 47, 17], np.int32)           # 47 == 47: nothing to do
    layout = W.scatter_pages(rng, lens)
    w = W.smoothing_weight(rng) if smooth else None
    if bits == 4:
        k, v = R.fill(rng, layout, lens, Hkv, w)
        src = pk.Pool(dev(k), dev(v))
        with np.errstate(invalid="ignore"):
            vals = [R.values(x).astype(np.float32) for x in (k, v)]      # exact in fp32
    else:
        shape = (layout.num_pages, Hkv, 16, 128)
        k, v = (rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2))
        ks, vs = (rng.uniform(0.001, 3, shape[:3]).astype(np.float32) for _ in range(2))
        src = pk.Pool(dev(k), dev(v), dev(ks), dev(vs))
        vals = [c.astype(np.float32) * s[..., None] for c, s in ((k, ks), (v, vs))]
    for st in (None, starts):
        s = np.zeros_like(lens) if st is None else st
        wide_bt, n = wide_layout(rng, lens, s)
        dst = pk.Pool(*(dev_bf16(np.full((n, Hkv, 16, 128), 0x1234, np.uint16)) for _ in range(2)))
        pk.kv_unpack(src, dst, dev(layout.block_table), dev(wide_bt), dev(lens), int(lens.max()),
                     starts=None if st is None else dev(st),
                     k_smooth=None if w is None else dev(w))
        assert pk.poll_device_error() == pk.OK
        for got, val, ww in ((dst.k, vals[0], w), (dst.v, vals[1], None)):
            want = expected_unpack(val, ww, layout.block_table, wide_bt, lens, s, n, 0x1234)
            assert np.array_equal(host_bits(got), want)


def test_unpack_flags_bad_tables_and_lengths(pk):
    rng = np.random.default_rng(930)
    lens = np.array([20, 20], np.int32)
    layout = W.scatter_pages(rng, lens)
    k, v = R.fill(rng, layout, lens, 2)
    src = pk.Pool(dev(k), dev(v))
    wide_bt, n = wide_layout(rng, lens, [0, 0])

    def go(bt=layout.block_table, wbt=wide_bt, ln=lens, starts=None):
        dst = pk.Pool(*(dev_bf16(np.full((n, 2, 16, 128), 0x1234, np.uint16)) for _ in range(2)))
        pk.kv_unpack(src, dst, dev(bt), dev(wbt), dev(ln), 32, starts=starts)
        return dst, pk.poll_device_error()

    for bad in ((0, -1), (0, layout.num_pages)):
        bt = layout.block_table.copy()
        bt[bad[0], 0] = bad[1]
        dst, st = go(bt=bt)
        assert st == pk.ERR_INVALID
        assert (host_bits(dst.k)[wide_bt[0, 0]] == 0x1234).all()         # skipped
        assert not (host_bits(dst.k)[wide_bt[1, 0]] == 0x1234).any()     # the others are done
    wbt = wide_bt.copy()
    wbt[1, 1] = n
    assert go(wbt=wbt)[1] == pk.ERR_INVALID
    assert go(ln=np.array([20, 33], np.int32))[1] == pk.ERR_INVALID      # past max_seq_len
    assert go(ln=np.array([20, -1], np.int32))[1] == pk.ERR_INVALID
    assert go(starts=dev(np.array([-1, 0], np.int32)))[1] == pk.ERR_INVALID
    assert go()[1] == pk.OK


@pytest.mark.parametrize("smooth", [False, True])
def test_chunked_prefill_against_a_4bit_prefix(pk, smooth):
    """The run of a prompt: its chunks are appended to the 4-bit pool, the new
    positions unpacked into bf16 pages, and each chunk attends to all of them;
    against float64 attention over the dequantised cache.  Measured
    against the bf16 pages' own values, the bars are the prefill tests'."""
    rng = np.random.default_rng(940)
    T, Hq, Hkv, chunk = 300, 8, 2, 128
    w = W.smoothing_weight(rng) if smooth else None
    layout = W.scatter_pages(rng, [T])
    bt = dev(layout.block_table)
    pool = pk.Pool.empty(layout.num_pages, Hkv, dtype=torch.uint8)
    wide_bt, n = wide_layout(rng, [T], [0])
    wide = pk.Pool.empty(n, Hkv)
    kn = W.keys_with_channel_weight(rng, (T, Hkv, 128), w) if smooth else W.normal_bf16(rng, (T, Hkv, 128))
    vn, q = W.normal_bf16(rng, (T, Hkv, 128)), W.normal_bf16(rng, (T, Hq, 128))
    ws = pk.prefill_workspace()
    kw = dict(k_smooth=None if w is None else dev(w))
    outs, lses = [], []
    for c in range(0, T, chunk):
        e = min(T, c + chunk)
        lens, cu = dev(np.array([e], np.int32)), dev(W.cu_from_counts([e - c]))
        pk.kv_append(pool, dev_bf16(kn[c:e]), dev_bf16(vn[c:e]), cu, bt, lens, **kw)
        pk.kv_unpack(pool, wide, bt, dev(wide_bt), lens, e, starts=dev(np.array([c], np.int32)), **kw)
        o, l = pk.paged_attn_prefill(wide, dev_bf16(q[c:e]), cu, dev(wide_bt), lens, e - c,
                                     128 ** -0.5, workspace=ws)
        outs.append(o)
        lses.append(l)
    assert pk.poll_device_error() == pk.OK
    import oracle
    from tests.helpers import check_lse, check_out
    ro, rl = oracle.paged_attention(host_bits(wide.k), host_bits(wide.v), q, [0, T], wide_bt,
                                    np.array([T], np.int32), 128 ** -0.5)
    check_out(torch.cat(outs), ro, "chunked prefill")
    check_lse(torch.cat(lses), rl, "chunked prefill")
    fo, _, _ = R.attention(pool.k.cpu().numpy(), pool.v.cpu().numpy(),
                        W.bits_to_float(q).astype(np.float64), [0, T], layout.block_table, [T],
                        128 ** -0.5, w)
    # bf16 pages: a score is off by at most eps = 2^-9 scale sum|q k|, so every p and the sum of
    # them by a factor within exp(+-eps); V is off by 2^-9 of itself; then the prefill's own bars
    kq = np.abs(R.values(pool.k.cpu().numpy())[layout.block_table[0]])
    kq = kq.transpose(1, 0, 2, 3).reshape(Hkv, -1, 128)[:, :T]
    kq = kq * w if smooth else kq
    aq = np.abs(W.bits_to_float(q)).reshape(T, Hkv, Hq // Hkv, 128)
    eps = 2.0 ** -9 * 128 ** -0.5 * np.einsum("thgd,hnd->thgn", aq, kq).max()
    vq = R.values(pool.v.cpu().numpy())[layout.block_table[0]]         # the cached positions alone
    vmax = np.abs(vq.transpose(1, 0, 2, 3).reshape(Hkv, -1, 128)[:, :T]).max()
    got = torch.cat(outs).float().cpu().numpy()
    assert np.abs(got - fo).max() <= np.expm1(2 * eps) * vmax + 2.0 ** -9 * vmax + 1e-2 * (1 + vmax)

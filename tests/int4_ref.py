"""The 4-bit cache in numpy: the quantiser's IEEE fp32 steps, the slab layout,
and attention over the dequantised values in float64.  Test infrastructure; it
shares no code with the library."""
import numpy as np

from paged_kv_flash_gb300 import workloads as W

SLAB = 1152


def quantize(x):
    """x fp32 [..., 128] -> (codes int [..., 128], fp16 scales [..., 4])."""
    g = np.asarray(x, np.float32).reshape(*x.shape[:-1], 4, 32)
    with np.errstate(all="ignore"):
        amax = np.abs(g).max(-1)                                     # NaN stays NaN
        s = np.minimum(amax / np.float32(7), np.float32(65504)).astype(np.float16)
        s = np.where(np.isfinite(amax), s, np.float16(np.nan))
        f = s.astype(np.float32)[..., None]
        c = np.clip(np.rint(g / f), -7, 7)
    c = np.where((f > 0) & np.isfinite(f), c, 0)
    return c.reshape(x.shape).astype(np.int64), s


def slab_row(codes, scales):
    """The bytes of one position: codes [..., 128], scales [..., 4] -> the 64
    code bytes [..., 4, 16] and the 8 scale bytes [..., 8]."""
    u = (codes + 8).astype(np.uint8).reshape(*codes.shape[:-1], 4, 16, 2)
    return u[..., 0] | (u[..., 1] << 4), np.ascontiguousarray(scales).view(np.uint8)


def put(pool, page, head, slot, codes, scales):
    """Write one vector into pool uint8 [pages][heads][1152]."""
    b, s = slab_row(codes, scales)
    for g in range(4):
        at = 256 * g + 16 * slot
        pool[page, head, at:at + 16] = b[g]
    pool[page, head, 1024 + 8 * slot:1032 + 8 * slot] = s


def values(pool):
    """pool uint8 [pages][heads][1152] -> float64 [pages][heads][16][128]."""
    P, H = pool.shape[:2]
    b = pool[..., :1024].reshape(P, H, 4, 16, 16)
    out = np.empty((P, H, 16, 4, 16, 2))
    out[..., 0] = (b & 15).astype(np.float64).transpose(0, 1, 3, 2, 4) - 8
    out[..., 1] = (b >> 4).astype(np.float64).transpose(0, 1, 3, 2, 4) - 8
    with np.errstate(invalid="ignore"):                      # NaN scales of unwritten slots
        s = np.ascontiguousarray(pool[..., 1024:]).view(np.float16).astype(np.float64)
        return (out * s.reshape(P, H, 16, 4, 1, 1)).reshape(P, H, 16, 128)


def fill(rng, layout, lens, Hkv, w=None, poison=0xFF):
    """Pools whose cached positions hold quantised N(0,1) vectors (keys times w,
    stored divided by it); every other byte is `poison` (NaN scales)."""
    pools = []
    for key in (True, False):
        pool = np.full((layout.num_pages, Hkv, SLAB), poison, np.uint8)
        for b, n in enumerate(np.asarray(lens)):
            for lp in range(-(-int(n) // 16)):
                page = layout.block_table[b, lp]
                m = min(16, int(n) - 16 * lp)
                x = rng.standard_normal((Hkv, m, 128), dtype=np.float32)
                if key and w is not None:
                    x = W.bits_to_float(W.to_bf16_bits(x * w)).astype(np.float32) / w
                c, s = quantize(x)
                code, sc = slab_row(c, s)                            # [H][m][4][16], [H][m][8]
                pool[page, :, :1024].reshape(Hkv, 4, 16, 16)[:, :, :m] = code.transpose(0, 2, 1, 3)
                pool[page, :, 1024:].reshape(Hkv, 16, 8)[:, :m] = sc
        pools.append(pool)
    return pools


def attention(k_pool, v_pool, q, cu_q, block_table, seq_lens, scale, w=None):
    """Causal attention (bottom-right aligned) of q float [T][Hq][128] in
    float64: (out [T][Hq][128], natural-log lse [T][Hq], sum p |v| [T][Hq][128])."""
    T, Hq, _ = q.shape
    Hkv = k_pool.shape[1]
    G = Hq // Hkv
    out, lse, mag = np.zeros((T, Hq, 128)), np.full((T, Hq), -np.inf), np.zeros((T, Hq, 128))
    for b, L in enumerate(np.asarray(seq_lens)):
        L, t0, t1 = int(L), int(cu_q[b]), int(cu_q[b + 1])
        if L == 0 or t1 == t0:
            continue
        pages = block_table[b, :-(-L // 16)]
        k = values(k_pool[pages]).transpose(1, 0, 2, 3).reshape(Hkv, -1, 128)[:, :L]
        v = values(v_pool[pages]).transpose(1, 0, 2, 3).reshape(Hkv, -1, 128)[:, :L]
        if w is not None:
            k = k * w.astype(np.float64)
        for t in range(t0, t1):
            n = L - (t1 - t0) + (t - t0) + 1
            qt = q[t].astype(np.float64).reshape(Hkv, G, 128)
            s = np.einsum("hgd,hnd->hgn", qt, k[:, :n]) * scale
            m = s.max(-1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(-1, keepdims=True)
            out[t] = (np.einsum("hgn,hnd->hgd", p, v[:, :n]) / l).reshape(Hq, 128)
            mag[t] = (np.einsum("hgn,hnd->hgd", p, np.abs(v[:, :n])) / l).reshape(Hq, 128)
            lse[t] = (m + np.log(l)).reshape(Hq)
    return out, lse, mag

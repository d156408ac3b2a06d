"""Plain FP64 forms (numpy) of the router, the whole layer and the adapted
projection, with bounds on what the kernels' arithmetic may be off."""

import numpy as np

import oracle

U32 = 2.0 ** -24  # FP32 half step
U16 = 2.0 ** -11  # fp16 half step
UBF = 2.0 ** -8   # bfloat16 half step


def weight(codes, sf, gs, gran):
    """[N, K/2] codes, [N, K/gran] scale bytes, gs a number or None -> [N, K] float64."""
    v = oracle.e2m1_decode(oracle.unpack_fp4(codes))
    s = oracle.e4m3_decode(sf) if gran == 16 else oracle.ue8m0_decode(sf)
    return v * np.repeat(s, gran, axis=1) * (1.0 if gs is None else float(gs))


def fp4_tensor(rng, E, N, K, gran, lo=-8.0, hi=-2.0):
    import torch
    w = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    if gran == 16:
        s = np.exp2(rng.uniform(lo, hi, (E, N, K // 16))).astype(np.float32)
        sf = torch.from_numpy(s).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    else:
        sf = rng.integers(127 + int(lo), 128 + int(hi), (E, N, K // 32)).astype(np.uint8)
    return w, sf


def layer(x, ids, wts, w13, w13_sf, w13_gs, w2, w2_sf, w2_gs, gran, order, hrel):
    """(out, bound) [T, H]: sum over a token's experts, and how far a kernel may be from it that sums in FP32
    in any order, evaluates SwiGLU to a few ulp, rounds h to hrel relative and weighs with FP32 weights.
    x [T, H] float64; rows with an id of -1 in a place lack that term."""
    T, H = x.shape
    I = w2.shape[2] * 2
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(ids[ids >= 0]):
        t, j = np.nonzero(ids == e)
        W = weight(w13[e], w13_sf[e], None if w13_gs is None else w13_gs[e], gran)
        V = weight(w2[e], w2_sf[e], None if w2_gs is None else w2_gs[e], gran)
        a, aa = x[t] @ W.T, np.abs(x[t]) @ np.abs(W).T
        sl = slice(0, I) if order == "gate_up" else slice(I, 2 * I)
        su = slice(I, 2 * I) if order == "gate_up" else slice(0, I)
        with np.errstate(over="ignore"):
            g, u = a[:, sl], a[:, su]
            silu = g / (1 + np.exp(-g))
        dg, du = (H + 16) * U32 * aa[:, sl], (H + 16) * U32 * aa[:, su]
        h = silu * u
        # |silu'| <= 1.1; exp, division and products: 16 half steps
        dh = 1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du + (16 * U32 + hrel) * np.abs(h)
        dh += 2.0 ** -38 * np.max(np.abs(h), axis=1, keepdims=True)  # fp16's smallest steps
        y, ya = h @ V.T, np.abs(h) @ np.abs(V).T
        dy = dh @ np.abs(V).T + (I + 64) * U32 * ya
        wj = wts[t, j][:, None]
        out[t] += wj * y
        # the weights' own error (tests/test_gpu_gate.py) and the sums over experts
        bound[t] += np.abs(wj) * (dy + 1024 * U32 * np.abs(y))
    return out, bound


def project(x, w, w_sf, w_gs, gran, a=None, b=None, ids=None, scale=None):
    """(y, bound) [T, N]: W x + s B (A x), and how far a kernel may be from it that sums in FP32 in any order, keeps
    x to 2^-39 of its row's maximum and A x to 17 bits."""
    W = weight(w, w_sf, None if w_gs is None else w_gs[0], gran)
    K = x.shape[1]
    y, ya = x @ W.T, np.abs(x) @ np.abs(W).T
    bound = (K + 16) * U32 * ya + 2.0 ** -38 * np.max(np.abs(x), axis=1, keepdims=True) * np.abs(W).sum(1)[None, :]
    if a is not None:
        L, R = a.shape[:2]
        for l in range(L):
            t = np.nonzero(ids == l)[0]
            u, ua = scale[l] * (x[t] @ a[l].T), np.abs(scale[l]) * (np.abs(x[t]) @ np.abs(a[l]).T)
            du = (K + 16) * U32 * ua + 2.0 ** -17 * np.abs(u)
            y[t] += u @ b[l].T
            bound[t] += du @ np.abs(b[l]).T + (R + 16) * U32 * (np.abs(u) @ np.abs(b[l]).T)
    return y, bound + 8 * U32 * np.abs(y)

"""FP64 definition of linear attention with a decay for each key/value head, and of the
magnitudes its rounding errors scale with. Plain torch in 64 bits, token by token; shares no
code with the CUDA path.

  S_t = lam S_{t-1} + v_t k_t^T,  o_t[h] = scale S_t q_t[h],  lam = exp(log_decay[h // R])
"""
from __future__ import annotations

import torch


def linattn(q, k, v, log_decay, scale, init=None, lens=None):
    """q [T,H,K], k [T,Hk,K], v [T,Hk,V] packed sequences of the given lengths (one if None);
    init [nseq,Hk,V,K] or None. Returns a dict of float64 tensors:
      o [T,H,V], final [nseq,Hk,V,K];
      o_mag: sum over sources of lam^(t-s) sum_i |q_i k_i| |v| (and |S_0|), times scale;
      o_score: the same with |q.k| for sum_i |q_i k_i| and without S_0 (what an error in the
               score multiplies);
      s_mag: sum over sources of lam^(L-1-s) |v| |k| (and |S_0|)."""
    q, k, v = q.double(), k.double(), v.double()
    T, H, K = q.shape
    Hk, V = v.shape[1:]
    lens = [T] if lens is None else [int(n) for n in lens]
    assert sum(lens) == T
    lam = torch.exp(log_decay.double()).view(Hk, 1, 1)
    dev = q.device
    o, om, osc = (torch.zeros(T, H, V, dtype=torch.float64, device=dev) for _ in range(3))
    fin = torch.zeros(len(lens), Hk, V, K, dtype=torch.float64, device=dev)
    fmag = torch.zeros_like(fin)
    at = 0
    for s, n in enumerate(lens):
        S = torch.zeros(Hk, V, K, dtype=torch.float64, device=dev) if init is None else init[s].double().clone()
        M = S.abs()
        for t in range(at, at + n):
            kv = v[t][:, :, None] * k[t][:, None, :]
            S = lam * S + kv
            M = lam * M + kv.abs()
            qt = q[t].view(Hk, H // Hk, K).transpose(1, 2)          # [Hk, K, R]
            o[t] = (S @ qt).transpose(1, 2).reshape(H, V) * scale
            om[t] = (M @ qt.abs()).transpose(1, 2).reshape(H, V) * abs(scale)
        # sum over sources of lam^(t-s) |q_t.k_s| |v_s|, quadratically
        if n:
            kk, vv = k[at:at + n], v[at:at + n].abs()
            qq = q[at:at + n].view(n, Hk, H // Hk, K)
            i = torch.arange(n, device=dev)
            dec = torch.exp(log_decay.double()[:, None, None] * (i[:, None] - i[None]).clamp(min=0)) * (i[:, None] >= i[None])
            sc = torch.einsum("thrk,shk->hrts", qq, kk).abs() * dec[:, None]
            osc[at:at + n] = torch.einsum("hrts,shv->thrv", sc, vv).reshape(n, H, V) * abs(scale)
        fin[s], fmag[s] = S, M
        at += n
    return {"o": o, "final": fin, "o_mag": om, "o_score": osc, "s_mag": fmag}

"""How near gdn_replay_advance comes to the 64-bit values over several hundred tokens, beside the worst-case bounds of advance_ref.

Limit of the chunked form, as the root mean square of the errors over that of the values.  In a chunk a value passes through three
products ([K;Q] S^T, then E x or (M P) x, whose factors are made by another).  Their operands are exact (three bf16 terms), so what is left are
the additions in the tensor cores, which do not round to nearest: they lie below the sum by up to 2^-23 of it, half of that on
average, all to one side.  The terms come smallest first, so eight additions (a contraction of 128 in steps of 16) act on a full-size sum:
3 * 8 * 2^-24 = 1.4e-6, and the limit is 2^-19 = 1.9e-6.  Operands of two terms are off by up to 2^-16 each, some 2^-18 of the
values after a product: several times the limit (shown below in the plain form).
Token by token: (dk + 8) roundings of 2^-24, at random signs sqrt(136) 2^-24 = 7e-7 at the most of a step's; a state that
forgets within a few tokens adds few of them up."""
import numpy as np
import pytest
import torch

import advance_ref as R

BF, F32 = torch.bfloat16, torch.float32
LIMIT = 2.0 ** -19


def inputs(B, T, H, dk, dv, decay, device, seed=51):
    g = torch.Generator(device=device).manual_seed(seed)
    unit = torch.nn.functional.normalize

    def randn(*s):
        return torch.randn(*s, generator=g, device=device)

    q, k = (unit(randn(B, T, H, dk), dim=-1).to(BF) for _ in range(2))
    return (q, k, randn(B, T, H, dv).to(BF), -decay * torch.nn.functional.softplus(randn(B, T, H)), torch.sigmoid(randn(B, T, H)),
            0.1 * randn(B, H, dv, dk))


def exact(q, k, v, g, beta, S, scale):
    q, k, v, g, beta, S = (x.double() for x in (q, k, v, g, beta, S))
    out = torch.empty_like(v)
    for t in range(v.shape[1]):
        S = S * g[:, t].exp()[..., None, None]
        w = (v[:, t] - (S @ k[:, t, :, :, None])[..., 0]) * beta[:, t, :, None]
        S = S + w[..., None] * k[:, t, :, None]
        out[:, t] = (S @ q[:, t, :, :, None])[..., 0] * scale
    return out, S


def rms(x):
    return x.double().square().mean().sqrt().item()


def advance(q, k, v, g, beta, S, dtype):
    import speculative_decode_recurrent_gb300 as lib
    B, T, H, dv = v.shape
    dk = k.shape[-1]
    dims = lib.Dims(B=B, H=H, dk=dk, dv=dv, T=1, cap=2, threshold=1, n_slot=B, scale=dk ** -0.5,
                    in_dtype=lib.DTYPE_BF16 if dtype == BF else lib.DTYPE_F32)
    z = torch.zeros
    layer = lib.ReplayLayer(dims, dict(state=S.clone(), state_idx=None, buf_k=z(B, H, 2, dk, dtype=dtype), buf_v=z(B, H, 2, dv, dtype=dtype),
                                       buf_g=z(B, H, 2), buf_beta=z(B, H, 2), buf_len=z(B, dtype=torch.int32)))
    out = torch.empty(B, T, H, dv, device="cuda")
    layer.advance(q.to(dtype), k.to(dtype), v.to(dtype), g, beta, out)
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    return out, layer.t["state"]


@pytest.mark.gpu
@pytest.mark.parametrize("decay", [1.0, 1e-2, 1e-3])         # 0.8 a token on average; states that last for 100 and 1000 tokens
@pytest.mark.parametrize("B,T,H,dk,dv", [
    (1, 640, 4, 128, 128), (2, 600, 16, 128, 128),           # slices of 16 and of 32 columns
    (8, 600, 16, 128, 128), (16, 500, 16, 64, 128),          # heads
    (2, 500, 20, 64, 64), (3, 500, 16, 128, 64),
])
def test_chunked_form_is_near_the_exact_values(B, T, H, dk, dv, decay, cuda_ok):
    x = inputs(B, T, H, dk, dv, decay, "cuda")
    out, S = exact(*x, dk ** -0.5)
    got, state = advance(*x, BF)
    assert rms(got - out) <= LIMIT * rms(out) and rms(state - S) <= LIMIT * rms(S), (rms(got - out) / rms(out), rms(state - S) / rms(S))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,H,dk,dv", [(1, 1, 16, 128, 128), (3, 5, 4, 64, 64), (9, 17, 16, 128, 64), (2, 23, 32, 64, 128)])
def test_short_calls_keep_the_bound_of_single_tokens(B, T, H, dk, dv, dtype, cuda_ok):
    """Calls of any type that go token by token, against the bound of that kernel (bf16 keys and values are exact in fp32)."""
    x = inputs(B, T, H, dk, dv, 1.0, "cuda", seed=52)
    got, state = advance(*x, dtype)
    for b in range(B):
        o, S, norm, eff = R.advance(*(y[b].double().cpu().numpy() for y in (x[5], x[0], x[1], x[2], x[3], x[4])), dk ** -0.5)
        tol = R.advance_bound(norm, eff, dk, False)
        assert np.abs(state[b].double().cpu().numpy() - S).max() <= tol
        assert np.abs(got[b].double().cpu().numpy() - o).max() <= 1.01 * tol * dk ** -0.5


def terms(x, n):
    """x in n bf16 terms, 8 bits of the mantissa after the other, the last one rounded."""
    x, y = x.float(), torch.zeros_like(x, dtype=torch.float64)
    for i in range(n):
        t = x.bfloat16().float() if i == n - 1 else (x.view(torch.int32) & -65536).view(torch.float32)
        y, x = y + t.double(), x - t
    return y


def chunked(q, k, v, g, beta, S, scale, n):
    """The chunked form in 64 bits, its operands in n bf16 terms."""
    q, k, v, g, beta, S = (x.double() for x in (q, k, v, g, beta, S))
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], 64):
        K, Q, V, G, b = (x[0, c:c + 64].transpose(0, 1) for x in (k, q, v, g, beta))     # [H, C, ..]
        G = G.cumsum(-1)
        D = torch.exp((G[:, :, None] - G[:, None]).tril()).tril()
        A = ((K @ K.transpose(1, 2)) * D).tril(-1) * b[..., None]
        P = torch.linalg.inv(torch.eye(A.shape[1], dtype=torch.float64) + A) * b[:, None]
        M, F = terms(scale * (Q @ K.transpose(1, 2)) * D, n), terms(P * torch.exp(G[:, -1:] - G)[..., None], n)
        E, MP, T = terms(K.transpose(1, 2) @ F, n), terms(M @ terms(P, n), n), terms(S, n)[0]
        x = terms(V - torch.exp(G)[..., None] * (K @ T.transpose(1, 2)), n)
        out[0, c:c + 64] = (scale * torch.exp(G)[..., None] * (Q @ T.transpose(1, 2)) + MP @ x).transpose(0, 1)
        S = (torch.exp(G[:, -1])[:, None, None] * S[0] + (E @ x).transpose(1, 2))[None]
    return out, S


def test_two_terms_would_not_pass():
    """The limit tells two terms from three: plain products in 64 bits of operands so rounded."""
    x = inputs(1, 192, 2, 128, 128, 1.0, "cpu", seed=53)
    out, S = exact(*x, 128 ** -0.5)
    for n, passes in ((2, False), (3, True)):
        o, s = chunked(*x, 128 ** -0.5, n)
        assert (rms(o - out) <= LIMIT * rms(out)) == passes, (n, rms(o - out) / rms(out), rms(s - S) / rms(S))

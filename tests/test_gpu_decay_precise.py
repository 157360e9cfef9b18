"""How many bits the states of decay attention keep: what the worst-case bounds of the other
tests are too wide for.  u = 2^-24, half a step of 32 bits.

A key times its weight goes into the tensor cores as three bf16 terms; two would leave up
to 2^-18 of it, and one 2^-9.  A state is multiplied by one power for every chunk, as two
floats; in one float its rounding would add up over the chunks."""
import math

import numpy as np
import pytest
import torch

import flash_mixed_chunk_gb300 as fm
from oracle import serve

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
# bf16 on the tensor cores (one and two blocks of keys), bf16 and fp32 on the CUDA cores
FORMS = [(BF16, 64, 64), (BF16, 128, 72), (BF16, 37, 20), (F32, 64, 40)]


def settled():
    torch.cuda.synchronize()
    assert fm.flash_mca_device_status()[0] == fm.FMCA_OK


def two_terms(x):
    """What two bf16 terms hold of fp32 values."""
    t0 = x.to(BF16).float()
    return t0.double() + (x - t0).to(BF16).double()


def wild_rates(H, seed=0):
    """Half-lives of 4 to 400 tokens: powers with all their bits in use."""
    g = torch.Generator().manual_seed(seed)
    return -math.log(2) / (4 * 100 ** torch.rand(H, generator=g))


@pytest.mark.parametrize("T", [20, 128, 500, 2600])
@pytest.mark.parametrize("dtype,dk,dv", FORMS)
def test_one_product_keeps_its_bits(dtype, dk, dv, T):
    """One token with a key: each place of the state is one product, lam^n k v.

    Roundings: the power (exp2f's two steps of 2 u, its correction u), the weighted key u,
    the terms' rest u / 4, the products' sum (cut, not rounded) 2 u and a little, and one u
    for every chunk behind it (32 or 128 tokens); where the sequence is cut, a segment's
    power 5 u and its addition u."""
    H = 16
    g = torch.Generator().manual_seed(T)
    ld = wild_rates(H, T)
    q, k, v = (torch.randn(1, T, H, d, generator=g).to(dtype) for d in (dk, dk, dv))
    at = [(7 * h + T // 2) % T for h in range(H)]
    at[0], at[1], at[2] = 0, T - 1, T - 2
    # no further back than 60 half-lives, so that nothing is under the normal range
    at = [max(t, T - 1 - int(60 * math.log(2) / -float(r))) for t, r in zip(at, ld)]
    keep = torch.zeros(1, T, H, 1)
    for h, t in enumerate(at):
        keep[0, t, h] = 1
    k = (k.float() * keep).to(dtype)
    o, s = fm.decay_attention(q.cuda(), k.cuda(), v.cuda(), ld.cuda())
    settled()
    s = s.double().cpu()[0]
    for h, t in enumerate(at):
        key, val = k[0, t, h].double(), v[0, t, h].double()
        w = math.exp(float(ld[h].double()) * (T - 1 - t))
        want = w * key[:, None] * val[None]
        tol = (8.5 + (T - 1 - t) // 32 + 2 + 6) * U
        assert ((s[h] - want).abs() <= tol * want.abs()).all(), (h, t)
    # the bound tells three terms from two, for keys whose weight is not a power of 2
    rest = []
    for h, t in enumerate(at):
        if 0 < (T - 1 - t) < 120:
            x = k[0, t, h].float() * float(np.float32(math.exp(float(ld[h]) * (T - 1 - t))))
            y = x[x != 0]
            rest.append(float(((two_terms(y) - y.double()) / y.double()).abs().max()))
    assert dtype == F32 or max(rest) > 1.3 * (8.5 + 120 // 32 + 8) * U


@pytest.mark.parametrize("T", [128, 390, 1100])
@pytest.mark.parametrize("dtype,dk,dv", FORMS)
def test_the_states_error_is_that_of_32_bits(dtype, dk, dv, T):
    """Root mean square error of the state, against that of the same sum from two bf16 terms
    of each weighted key: under half of it (for fp32 operands too).  An emulation of sums cut
    after every 16 tokens of every term stays under a quarter."""
    H = 6
    g = torch.Generator().manual_seed(T + dk)
    ld = wild_rates(H, T)
    q, k, v = (torch.randn(1, T, H, d, generator=g).to(dtype) for d in (dk, dk, dv))
    s0 = torch.randn(1, H, dk, dv, generator=g)
    _, s = fm.decay_attention(q.cuda(), k.cuda(), v.cuda(), ld.cuda(), state=s0.cuda())
    settled()
    _, want, _ = serve.decay_attention(q, k, v, ld, s0)
    err = (s.cpu().double() - torch.as_tensor(want))[0]
    for h in range(H):
        w = torch.exp(ld[h].double() * (T - 1 - torch.arange(T))).float()[:, None]
        x = k[0, :, h].float().to(BF16).float() * w
        less = (two_terms(x) - x.double()).T @ v[0, :, h].double()
        rms = lambda e: float(e.pow(2).mean().sqrt())  # noqa: E731
        assert rms(err[h]) <= 0.5 * rms(less), (h, rms(err[h]), rms(less))


@pytest.mark.parametrize("dtype,d,chunk", [(BF16, 16, 128), (F32, 8, 32), (BF16, 9, 32)])
def test_many_chunks_powers_do_not_add_up(dtype, d, chunk):
    """A carried state alone, uncut: lam^T S.  Each chunk rounds each place anew (up to u,
    evenly to both sides), but its power must not be off by the same every time.  So the mean
    error of N places after G chunks is that of N G roundings, sqrt(G / (3 N)) u, and G times
    what two floats leave (2^-30); one float's rounding of the power would be G times that."""
    H, G = 480, 150
    T = G * chunk
    # a rate whose power of a chunk is off by over u / 3 in one float, and kept by two thirds
    for i in range(1000):
        ld = torch.tensor(-0.4 / T * (1 + i / 1000), dtype=F32)
        p = math.exp(float(ld) * chunk)
        off = float(np.float32(p)) / p - 1
        if abs(off) > U / 3:
            break
    assert abs(off) > U / 3
    g = torch.Generator().manual_seed(d)
    s0 = torch.randn(1, H, d, d, generator=g).cuda()
    z = torch.zeros(1, T, H, d, dtype=dtype, device="cuda")
    lds = torch.full((H,), float(ld), device="cuda")
    _, s = fm.decay_attention(z, z, z, lds, state=s0)
    settled()
    want = s0.double() * math.exp(float(ld) * T)
    mean = float(((s.double() - want) / want).mean())
    N = s0.numel()
    limit = 6 * math.sqrt(G / (3 * N)) * U + G * 2.0 ** -30
    assert limit < 0.5 * G * abs(off)
    assert abs(mean) <= limit, (mean, limit)
    tol = (G + 1) * 1.01 * U + G * 2.0 ** -30
    assert ((s.double() - want).abs() <= tol * want.abs()).all()

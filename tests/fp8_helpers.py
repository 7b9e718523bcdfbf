"""64-bit definitions and inputs of the 8-bit operators, for their tests."""
import torch

G = 128
F8 = torch.float8_e4m3fn
TINY = 2.0 ** -126


def groups(n):
    return -(-n // G)


def expand(scales, n):
    """[.., groups] scales as [.., n] columns."""
    return scales.double().repeat_interleave(G, -1)[..., :n]


def quantize64(v):
    """Scales, and the values v / scale that 8 bits round."""
    rows, n = v.shape
    s = torch.empty((rows, groups(n)), dtype=torch.float64, device=v.device)
    for g in range(groups(n)):
        s[:, g] = v[:, g * G:(g + 1) * G].abs().amax(1) / 448
    return torch.where(s < TINY, TINY, s)


def strided(rows, columns, dtype, pad, device="cuda", lead=0):
    """An uninitialised [rows, columns] view whose rows are columns + pad apart, `lead` elements into its buffer."""
    raw = torch.empty(rows * (columns + pad) + lead, dtype=torch.uint8 if dtype == F8 else dtype, device=device)
    if dtype == F8:
        raw.fill_(0x7f)                      # NaN: whatever is read outside the rows shows
        raw = raw.view(F8)
    else:
        raw.fill_(float("nan"))
    return raw[lead:].view(rows, columns + pad)[:, :columns]


def f8_rows(rows, k, gen, pad=0, scale=1.0):
    """Random 8-bit rows over the whole range of values, padded so that rows start on 16 bytes, with scales."""
    ld = -(-(k + pad) // 16) * 16
    x = strided(rows, k, F8, ld - k)
    v = torch.randn((rows, k), generator=gen, device="cuda") * 40
    x.copy_(v.clamp(-448, 448).to(F8))
    s = torch.rand((rows, groups(k)), generator=gen, device="cuda") * scale + 0.01 * scale
    return x, s


def f8_weight(n, k, gen, experts=None, pad=0):
    e = experts or 1
    x, _ = f8_rows(e * n, k, gen, pad)
    s = (torch.rand((e, groups(n), groups(k)), generator=gen, device="cuda") + 0.01) / (k ** 0.5 * 1000)
    x = x.as_strided((e, n, k), (n * x.stride(0), x.stride(0), 1))
    return (x, s) if experts else (x[0], s[0])


def product64(x, xs, w, ws):
    """y and the bound of its fp32 summation error, both [rows, N] in 64 bits.

    In a group the tensor cores add 128 exact products in fp32 (each addition may truncate: 2^-23 of the sum of
    magnitudes at most), then a scale product (two roundings), and the groups are added."""
    a = x.double() * expand(xs, x.shape[1])
    k, n = w.shape[1], w.shape[0]
    b = w.double() * expand(ws, k).repeat_interleave(G, 0)[:n]
    return a @ b.t(), (a.abs() @ b.abs().t()) * ((G + groups(k) + 4) * 2.0 ** -23)


def assert_bf16_close(got, ref, bound, what=""):
    """got: bf16 roundings of values within `bound` of ref (8 significant bits: half a unit is up to 2^-8 of the value)."""
    g = got.double()
    assert torch.isfinite(g).all(), what
    off = (g - ref).abs() - (bound + 2.0 ** -8 * (ref.abs() + bound) + 2.0 ** -133)
    assert (off <= 0).all(), "%s: %g over the bound" % (what, off.max().item())


def assert_f8_close(q, scales, v, s64, rel, what=""):
    """q and scales against v = the 64-bit row, whose own error is rel * |v| at most: the nearest 8-bit value is within
    2^-4 of the value, or half of the least step 2^-9 of the scale."""
    s = scales.double()
    assert ((s - s64).abs() <= (rel + 2.0 ** -22) * s64).all(), what + ": scales"
    n = v.shape[1]
    se = expand(scales, n)
    got = q.double() * se
    step = torch.maximum(v.abs() * 2.0 ** -4, se * 2.0 ** -10)
    off = (got - v).abs() - step * (1 + 1e-4) - v.abs() * (2 * rel + 2.0 ** -20)
    assert (off <= 0).all(), "%s: q %g over the bound" % (what, off.max().item())

"""Rotary positions on the way into the cache, against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cascade_gb300 as pkc
import prompt_reference as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def workspace():
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    pkc.workspace_init(ws)
    return ws


def e4m3_values():
    return torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()


class Case:
    def __init__(self, T, hq, hkv, dtype, kind, rot=128, page=16, far=5000, factor=1.0, seed=0, gap=0):
        gen = torch.Generator().manual_seed(seed)
        self.T, self.hq, self.hkv, self.dtype, self.kind = T, hq, hkv, dtype, kind
        heads = hq + 2 * hkv + gap
        qkv = torch.randn((T, heads, 128), generator=gen).to(dtype)
        self.host = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:hq + 2 * hkv]
        d = qkv.cuda()
        self.q, self.k, self.v = d[:, :hq], d[:, hq:hq + hkv], d[:, hq + hkv:hq + 2 * hkv]
        self.positions = torch.randint(0, far + 1, (T,), generator=gen, dtype=torch.int32)
        self.pages = -(-T // page) + 2
        self.page = page
        self.slots = torch.randperm(self.pages * page, generator=gen)[:T]
        self.freq, self.amp = pkc.rope_frequencies(rot, factor=factor, context=4096 if factor > 1 else None, device="cpu")
        self.k_scale, self.v_scale = (0.25, 0.0625) if kind == "e4m3" else (1.0, 1.0)
        self.ws = workspace()
        shape = (self.pages, page, hkv, 128)
        self.pools = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") if kind == "e4m3" else
                      torch.full(shape, math.nan, dtype=dtype, device="cuda") for _ in "kv"]

    def run(self, interleaved, **more):
        return pkc.rope_append_kv(self.q, self.k, self.v, self.positions.cuda(), self.slots.cuda(), self.freq.cuda(), *self.pools, self.ws,
                                  interleaved=interleaved, amplitude=self.amp, k_scale=self.k_scale, v_scale=self.v_scale, **more)

    def check(self, q_out, interleaved, rows=None):
        """Turned rows: float32 products and sum (three roundings of their terms, and 2^-21 of them for the angle,
        its sine and cosine: 2^-20 together), then half a step of the type."""
        half = ref.HALF_STEP[self.dtype]
        tokens = torch.arange(self.T) if rows is None else rows
        want, size = ref.rotate(self.host[0], self.positions, self.freq, interleaved, self.amp)
        off = (q_out.cpu().double() - want).abs() - (half * want.abs() + 2.0 ** -19 * size + 2.0 ** -25)
        assert float(off.max()) <= 0
        key, size = ref.rotate(self.host[1], self.positions, self.freq, interleaved, self.amp)
        val = self.host[2].double()
        for pool, x, s, scale in zip(self.pools, (key, val), (size, None), (self.k_scale, self.v_scale)):
            got = pool.cpu().reshape(-1, self.hkv, 128)
            err = torch.zeros_like(x) if s is None else 2.0 ** -19 * s
            if self.kind == "e4m3":
                got = e4m3_values()[got.long()]
                x, err = x / scale, err / scale + 2.0 ** -22 * x.abs() / scale
                x = x.clamp(-448, 448)
                step = torch.pow(2.0, torch.floor(torch.log2((x.abs() + err).clamp(min=2.0 ** -6))) - 3)
                err = err + step / 2
            elif s is None:
                assert torch.equal(got[self.slots[tokens]], self.host[2][tokens])
                continue
            else:
                err = err + half * x.abs() + 2.0 ** -25
            off = (got[self.slots[tokens]].double() - x[tokens]).abs() - err[tokens]
            assert float(off.max()) <= 0
        # every other slot as it was
        rest = torch.ones(self.pages * self.page, dtype=torch.bool)
        rest[self.slots[tokens]] = False
        for pool in self.pools:
            other = pool.reshape(-1, self.hkv, 128).cpu()[rest]
            assert (other == 0x7F).all() if self.kind == "e4m3" else other.isnan().all()
        assert pkc.device_status(self.ws) == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("T,hq,hkv,dtype,rot,page", [
    (1, 8, 8, F16, 128, 16), (3, 32, 8, BF16, 128, 16), (5, 4, 4, F16, 16, 5), (33, 8, 1, BF16, 96, 16), (130, 7, 3, F16, 64, 20),
    (1000, 32, 8, BF16, 128, 64), (5001, 2, 2, F16, 112, 8),
])
def test_rows(T, hq, hkv, dtype, rot, page, kind, interleaved):
    c = Case(T, hq, hkv, dtype, kind if kind == "e4m3" else "16", rot, page, seed=T)
    c.check(c.run(interleaved), interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_more_tokens_than_warps(interleaved):
    c = Case(20011, 4, 1, BF16, "16", seed=2)
    c.check(c.run(interleaved), interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("factor", [1.0, 8.0])
def test_far_positions(factor, interleaved):
    """Positions up to 2^31 - 1: the angle's own error is that of float64's product."""
    c = Case(64, 4, 2, F16, "16", far=2 ** 31 - 1, factor=factor, seed=7)
    c.positions[:3] = torch.tensor([2 ** 31 - 1, 2 ** 30, 0], dtype=torch.int32)
    # the reference's product is off by 2^-53 of up to 2^31 radians, the kernel's fraction by 2^-52 of as many: 2^-20.4 of a radian
    q = c.run(interleaved)
    want, size = ref.rotate(c.host[0], c.positions, c.freq, interleaved, c.amp)
    off = (q.cpu().double() - want).abs() - (2.0 ** -11 * want.abs() + (2.0 ** -19 + 2.0 ** -20) * size)
    assert float(off.max()) <= 0


def test_negative_positions_and_frequencies():
    """Turning by -p is turning back."""
    c = Case(40, 4, 2, F16, "16", seed=8)
    c.positions = -c.positions
    c.check(c.run(False), False)
    c = Case(40, 4, 2, F16, "16", seed=8)
    c.freq = -c.freq * 7.3
    c.check(c.run(True), True)


def test_dense_in_place_and_gap():
    c = Case(77, 8, 2, BF16, "16", gap=3, seed=3)
    c.check(c.run(False), False)
    c = Case(77, 8, 2, BF16, "16", seed=3)
    c.q = c.q.contiguous()
    out = c.run(True, q_out=c.q)
    assert out.data_ptr() == c.q.data_ptr()
    c.check(out, True)


def test_tokens_without_a_place():
    c = Case(50, 4, 2, F16, "16", seed=4)
    keep = torch.arange(50) % 3 != 0
    whole = c.slots.clone()
    c.slots = torch.where(keep, whole, torch.full_like(whole, -1))
    q = c.run(False)
    c.slots = whole
    c.check(q, False, rows=torch.arange(50)[keep])
    c.slots[1] = c.pages * c.page
    c.run(False)
    assert pkc.device_status(c.ws) == 4


def test_special_values():
    """Infinities and NaN stay in their pairs; e4m3 takes +-448 beyond its range and keeps NaN."""
    c = Case(4, 1, 1, F16, "e4m3", rot=32, seed=5)
    c.k = c.k.clone()
    c.v = c.v.clone()
    c.v[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 60000.0], dtype=F16)
    c.k[1, 0, 3] = math.nan
    c.k[2, 0, 40] = math.inf
    c.k, c.v = c.k, c.v
    c.run(True)
    vals = e4m3_values()
    k, v = (vals[p.cpu().reshape(-1, 1, 128).long()][c.slots] for p in c.pools)
    assert v[0, 0, :2].tolist() == [448.0, -448.0] and v[0, 0, 2].isnan() and float(v[0, 0, 3]) == 448.0
    assert k[1, 0].isnan().nonzero().flatten().tolist() == [2, 3]
    assert float(k[2, 0, 40]) == 448.0 and not k[2].isnan().any()


def test_refuses():
    c = Case(6, 4, 2, F16, "16")
    pos, slots, f = c.positions.cuda(), c.slots.cuda(), c.freq.cuda()
    with pytest.raises(ValueError, match="dense heads"):
        pkc.rope_append_kv(c.q.transpose(0, 1).contiguous().transpose(0, 1), c.k, c.v, pos, slots, f, *c.pools, c.ws)
    with pytest.raises(ValueError, match="same strides"):
        pkc.rope_append_kv(c.q, c.k, c.v.contiguous(), pos, slots, f, *c.pools, c.ws)
    with pytest.raises(TypeError, match="dtype"):
        pkc.rope_append_kv(c.q, c.k, c.v, pos.long(), slots, f, *c.pools, c.ws)
    with pytest.raises(TypeError, match="dtype"):
        pkc.rope_append_kv(c.q, c.k, c.v, pos, slots, f.float(), *c.pools, c.ws)
    with pytest.raises(TypeError, match="dtype"):
        pkc.rope_append_kv(c.q.bfloat16(), c.k.bfloat16(), c.v.bfloat16(), pos, slots, f, *c.pools, c.ws)
    with pytest.raises(pkc.PkcError):
        pkc.rope_append_kv(c.q, c.k, c.v, pos, slots, f[:12], *c.pools, c.ws)  # 24 elements
    with pytest.raises(pkc.PkcError):
        pkc.rope_append_kv(c.q, c.k, c.v, pos, slots, f, *c.pools, c.ws, k_scale=2.0)
    with pytest.raises(ValueError, match="shape"):
        pkc.rope_append_kv(c.q, c.k, c.v, pos[:5], slots, f, *c.pools, c.ws)


def nearest_codes(x):
    """The e4m3 values nearest to float64 x, ties to the even code, at most 448."""
    a = x.abs().clamp(max=448.0)
    step = torch.pow(2.0, torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign(torch.round(a / step) * step, x)


@pytest.mark.parametrize("dtype,scale", [(BF16, 224.0), (F16, 1632.0), (F16, 1312.0), (BF16, 0.25), (F16, 0.0371), (BF16, 3.3e-4), (F16, 2.0 ** -100)])
def test_codes_of_the_quotient(dtype, scale):
    """Every 16-bit value over the scale, as value and as the part of a key that is not turned: the code nearest to
    the float32 quotient.  350 / 224 lies between two codes, and so do other values that a rounded reciprocal moves."""
    scale = float(np.float32(scale))
    x = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(dtype).reshape(512, 1, 128)
    c = Case(512, 1, 1, dtype, "e4m3", rot=16, seed=6)
    c.k, c.v, c.k_scale, c.v_scale = x.cuda(), x.cuda(), scale, scale
    c.run(False)
    want = nearest_codes((x.float() / torch.tensor(scale)).double())
    for pool, cols in zip(c.pools, (slice(16, 128), slice(0, 128))):
        got = e4m3_values()[pool.cpu().reshape(-1, 1, 128)[c.slots].long()]
        assert torch.equal(got[..., cols].nan_to_num(nan=1000.0), want[..., cols].nan_to_num(nan=1000.0))


def test_outputs_beside_the_inputs():
    """q_out right before and right behind the projection, between two tokens' rows, and on the only token's query."""
    c = Case(9, 4, 2, BF16, "16", seed=9)
    buf = torch.zeros(9 * (8 + 4 + 4) * 128, dtype=BF16, device="cuda")
    rows = buf[9 * 4 * 128:9 * 12 * 128].view(9, 8, 128)
    rows[:, :4], rows[:, 4:6], rows[:, 6:] = c.q, c.k, c.v
    c.q, c.k, c.v = rows[:, :4], rows[:, 4:6], rows[:, 6:]
    c.check(c.run(False, q_out=buf[:9 * 4 * 128].view(9, 4, 128)), False)
    c.check(c.run(False, q_out=buf[9 * 12 * 128:].view(9, 4, 128)), False)
    c = Case(2, 4, 2, BF16, "16", seed=10, gap=8)
    gap = torch.as_strided(c.q, (2, 4, 128), (512, 128, 1), c.v.storage_offset() + 256)
    c.check(c.run(True, q_out=gap), True)
    c = Case(1, 4, 2, BF16, "16", seed=11)
    c.check(c.run(True, q_out=c.q), True)
    c = Case(2, 4, 2, BF16, "16", seed=11)
    with pytest.raises(pkc.PkcError, match="overlap"):
        pkc.rope_append_kv(c.q, c.k, c.v, c.positions.cuda(), c.slots.cuda(), c.freq.cuda(), *c.pools, c.ws,
                           q_out=torch.as_strided(c.q, (2, 4, 128), (512, 128, 1)))


@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_least_alignment(kind):
    """Rows and pools on 16 bytes, slots and frequencies on 8, positions on 4."""
    def shifted(x, by):
        buf = torch.zeros(x.numel() + 256 // x.element_size(), dtype=x.dtype, device="cuda")
        out = buf[by // x.element_size():][:x.numel()].view(x.shape)
        assert out.data_ptr() % 256 == by
        return out.copy_(x)

    c = Case(61, 4, 2, F16, kind, rot=64, seed=12)
    rows = shifted(torch.cat(c.host, 1), 16)
    c.q, c.k, c.v = rows[:, :4], rows[:, 4:6], rows[:, 6:]
    c.pools = [shifted(p, by) for p, by in zip(c.pools, (16, 48))]
    out = pkc.rope_append_kv(c.q, c.k, c.v, shifted(c.positions, 4), shifted(c.slots, 8), shifted(c.freq, 8), *c.pools, c.ws, amplitude=c.amp,
                             k_scale=c.k_scale, v_scale=c.v_scale, q_out=shifted(torch.zeros((61, 4, 128), dtype=F16), 16))
    c.check(out, False)

"""Codes of the 8-bit quantisation where its quotients are hardest to round."""
import pytest
import torch

import bit_rank_post_amd as tq
from tests.gpu_util import need_gpu
from tests.ops_util import gen
from tests.test_gpu_fp8 import E4M3, quant_rows_ref, ref_scale

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    need_gpu()


def quantise(x):
    q = torch.zeros(x.shape, dtype=E4M3, device="cuda")
    c = torch.zeros((x.shape[0], -(-x.shape[1] // 128)), device="cuda")
    tq.fp8_quant_rows(x.cuda(), q, c)
    return q.cpu(), c.cpu()


def border_rows(e, n, g):
    """Rows with a scale of exponent e whose significand lies next to 1 or 2
    (there the quotients are closest to the middle of two f32 values), with
    values next to the borders between two codes."""
    near = torch.arange(n // 2).float() * 2.0 ** -23
    c = torch.cat([1 + near, 2 - 2.0 ** -23 - near])[:, None].double() * 2.0 ** e
    code = torch.randint(0, 40, (n, 128), generator=g).double()
    man, exp = code % 8, torch.floor(code / 8)
    val = torch.where(exp > 0, (1 + (man + 0.5) / 8) * torch.exp2(exp - 7), (man + 0.5) * 2.0 ** -9)
    x = (val * c).float()
    step = torch.randint(-2, 3, x.shape, generator=g, dtype=torch.int32)
    x = (x.view(torch.int32) + step).view(torch.float32)
    x[:, 0] = (c[:, 0] * 448).float()
    return x


@pytest.mark.parametrize("e", [-126, -101] + list(range(-100, -86)) + [0, 118])
def test_codes_at_every_size_of_scale(e):
    print(f"[case] codes at scales of 2^{e}", flush=True)
    x = border_rows(e, 256, gen(20 + e))
    q, c = quantise(x)
    rq, rc = quant_rows_ref(x)
    assert torch.equal(c, rc)
    wrong = q.float().double() != rq
    assert not wrong.any(), f"{int(wrong.sum())} codes, e.g. {x[wrong][0].item().hex()} at {c[wrong.any(1)][0].item().hex()}"


@pytest.mark.parametrize("amax,v", [("0x1.c0000ap-92", "0x1.800008p-109"), ("0x1.f7fffep-90", "0x1.9dfffcp-104"),
                                    ("0x1.bffffep-85", "0x1p-103")])
def test_quotients_next_to_a_border(amax, v):
    """Single quotients within 2^-24 of a border between two codes."""
    x = torch.zeros((1, 128))
    x[0, 0], x[0, 1] = float.fromhex(amax), float.fromhex(v)
    q, c = quantise(x)
    rq, rc = quant_rows_ref(x)
    assert torch.equal(c, rc) and torch.equal(c, ref_scale(x.abs().amax(1, keepdim=True)))
    assert torch.equal(q.float().double(), rq)


@pytest.mark.parametrize("amax", [1.0, 2.0 ** -110])
def test_zeros_keep_their_sign(amax):
    """-0 / c is -0, and so is what rounds to zero from below."""
    x = torch.zeros((1, 128))
    x[0, :6] = torch.tensor([amax, -0.0, 0.0, -amax * 2.0 ** -21, amax * 2.0 ** -21, -amax])
    want = torch.tensor([0x7E, 0x80, 0x00, 0x80, 0x00, 0xFE], dtype=torch.uint8)
    q, _ = quantise(x)
    assert torch.equal(q.view(torch.uint8)[0, :6], want)
    w = x.cuda()
    q, c = torch.zeros((1, 128), dtype=E4M3, device="cuda"), torch.zeros((1, 1), device="cuda")
    tq.fp8_quant_blocks(w, q, c)
    assert torch.equal(q.cpu().view(torch.uint8)[0, :6], want)

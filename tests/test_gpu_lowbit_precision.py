"""What attention over the low-bit caches may lose of small rows beside large and zero ones (bounds: lowbit_precision.py)."""
import pytest
import torch

from gpu_helpers import gpu, lib_ready
from lowbit_cases import quantise4
from lowbit_precision import Rows

pytestmark = gpu
FULL = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("power", [0, -10])
@pytest.mark.parametrize("split", [False, True])
def test_decode_zero_rows_set_no_unit(bits, power, split):
    """A zero V row has the scale 1 (the exponent 2^0 in 4 bits), far above that of rows of ordinary size: they must keep
    their weights' bits.  Every head pair has one head that looks at a single key and one that looks at many."""
    c = Rows([1500, 700, 33] if split else [700] * 40, [1] * (3 if split else 40), FULL, 0, 61, bits)
    c.v_host *= 2.0 ** power
    c.v_host[:, 3::17] *= 0
    c.v_host[:, 100:140] *= 0                    # a whole warp's share
    c.upload()
    c.aim(range(0, 32, 2), lambda s, p: (p * 7 // 11) | 1)
    c.compare(False, f"2^{power}")


@pytest.mark.parametrize("bits", [8, 4])
def test_decode_of_zero_rows_alone(bits):
    c = Rows([600, 40], [1, 1], FULL, 0, 63, bits)
    c.v_host *= 0
    c.upload()
    c.qd = c.q.cuda()
    out, lse = c.call(False)
    assert (out == 0).all() and lse.isfinite().all()


BITS = pytest.mark.parametrize("bits", [8, 4])
# (context lengths, new tokens) by the form that the prefill takes: keys of a unit split over a cluster, pairs of CTAs
# (more units of 64 than half of the SMs), pairs in a planned order (more pairs than half of the SMs), a CTA a unit
# (64 tokens at most), the same in a planned order (more units than SMs)
FORMS = {"split": ([1500], [40]), "pairs": ([1100, 900, 700, 650, 1030], [128, 100, 65, 77, 90]),
         "planned pairs": ([900 + 13 * i for i in range(10)], [128 - 5 * i for i in range(10)]),
         "one": ([900 + 13 * i for i in range(10)], [64 - 5 * i for i in range(10)]),
         "planned": ([900 - 13 * i for i in range(20)], [64 - 3 * i for i in range(20)])}
FORM = pytest.mark.parametrize("form", FORMS)


def near(s, p):
    return (p * 5 // 7) | 1


@BITS
@FORM
def test_prefill_small_rows_beside_zero_rows(bits, form):
    """V rows of 2^-14 beside zero rows, whose scale of 1 sets the unit: they enter as f16 of what they stand for."""
    c = Rows(*FORMS[form], FULL, 0, 65, bits)
    c.v_host *= 2.0 ** -14
    c.v_host[:, 4::18] *= 0
    c.upload()
    c.aim(range(0, 32, 2), near)
    c.compare(True, form)


@BITS
@FORM
def test_prefill_rows_of_2_to_the_minus_13_of_the_unit(bits, form):
    """Weights almost wholly on V rows 2^-8 to 2^-13 of the largest beside them."""
    c = Rows(*FORMS[form], FULL, 0, 67, bits)
    g = torch.Generator().manual_seed(2)
    power = torch.randint(-13, -7, c.v_host.shape[:2], generator=g).float()
    power[:, 4::18] = 0
    c.v_host *= torch.exp2(power)[..., None, None].to(torch.bfloat16)
    c.upload()
    c.aim(range(0, 32, 2), near)
    c.compare(True, form)


def test_decode_rows_of_2_to_the_minus_13_of_the_unit():
    c = Rows([1500, 700], [1, 1], FULL, 0, 69)
    power = torch.randint(-13, -7, c.v_host.shape[:2], generator=torch.Generator().manual_seed(2)).float()
    power[:, 4::18] = 0
    c.v_host *= torch.exp2(power)[..., None, None].to(torch.bfloat16)
    c.upload()
    c.aim(range(0, 32, 2), near)
    c.compare(False, "decode")


@BITS
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("q_len", [40, 128])
def test_prefill_rows_that_a_token_does_not_see(bits, which, q_len):
    """A sequence's last row, 2^20 times the others, is in the unit of tokens that do not see it: they lose 2^-25 of
    the unit, 2^-33 of that row, and no more."""
    lens = [700] * 10
    c = Rows(lens, [q_len] * 10, FULL, 0, 71, bits)
    host = c.k_host if which == "k" else c.v_host
    for s, n in enumerate(lens):
        host[c.table[s, (n - 1) // 256] - c.far, (n - 1) % 256] *= 2.0 ** 20
    c.upload()
    c.aim(range(0, 32, 2), near)
    c.compare(True, which)


def growths(tops, headroom):
    """How often the unit of V is taken anew over these key tiles' largest exponents (None: no row with one)."""
    sigma, n = None, 0
    for top in tops:
        if top is not None and (sigma is None or top > sigma + headroom):
            n += sigma is not None
            sigma = top
    return n


@pytest.mark.parametrize("bits,first", [(8, "unset"), (8, "zero"), (8, "small"), (4, "zero"), (4, "small")])
@FORM
def test_prefill_unit_of_v_grows(bits, first, form):
    """V rows 2^9 larger from key tile to key tile (every fourth falls back by 2^30), so that the unit of V is taken anew and O
    rescaled.  The first tile: small rows, zero rows with the appends' scale 1, or zero rows under the scale 0, which set no
    unit."""
    lens, q_lens = FORMS[form]
    c = Rows(lens, q_lens, FULL, 0, 73, bits)
    start = -60 if first != "zero" else 0
    for s, n in enumerate(lens):
        for b in range(0, n, 128):
            t = b // 128
            rows = c.v_host[c.table[s, b // 256] - c.far, b % 256:b % 256 + 128]
            rows *= 0 if t == 0 and first != "small" else 2.0 ** (start + 9 * t - (30 if t % 4 == 3 else 0))
    c.upload()
    if first == "unset":
        for s in range(len(lens)):
            c.pools[3][c.bt[s, 0].long(), :, :128] = 0.0
    c.aim(range(0, 32, 2), near)
    # every unit's list of tiles, and where CTAs share it some run of each way to do so, takes the unit anew
    headroom = 7 if bits == 8 else 4
    for s, (m, n) in enumerate(zip(q_lens, lens)):
        for h in range(8):
            tops = []
            for b in range(0, n, 128):
                rows = c.v[s][b:b + 128, h].abs().amax(-1)
                if bits == 8:
                    rows = torch.where(rows == 0, 0.0 if first == "unset" else 1.0, rows / 448)
                    tops.append(int(torch.frexp(rows.max())[1]) if rows.max() > 0 else None)
                else:
                    tops.append(int(quantise4(c.v[s][b:b + 128, h])[2].max()) - 127)
            assert growths(tops, headroom) >= 1
            if form == "split":
                for ctas in range(2, 9):
                    run = -(-len(tops) // ctas)
                    assert any(growths(tops[i:i + run], headroom) for i in range(0, len(tops), run))
    c.compare(True, form)

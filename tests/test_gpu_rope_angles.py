"""The angles of rotary positions at far positions, against whole-number arithmetic."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BITS = 300  # of 1 / 2 pi


def inverse_two_pi():
    """floor(2^BITS / 2 pi), pi by Machin's formula."""
    one = 1 << (BITS + 40)

    def arctan_inverse(n):
        term, total, k = one // n, 0, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total
    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    return (one << BITS) // (2 * pi)


def turns(p, f, inv):
    """p f / 2 pi less whole turns, in [0, 1), exact but for a rounding to a double."""
    num, den = float(f).as_integer_ratio()          # den is a power of two
    x = p * num * inv                                # over den 2^BITS
    shift = den.bit_length() - 1 + BITS
    return ((x % (1 << shift)) >> (shift - 60)) / 2.0 ** 60


@pytest.mark.parametrize("rotary,base", [(128, 1e4), (128, 5e5), (128, 1e7), (64, 5e5)])
def test_angles_at_far_positions(rotary, base):
    """|p| 2^-65 turns and what the cosines of angles within a turn are off by (test_gpu_rope's turned_bound): 2^-22."""
    import paged_kv_cache_306_gb300 as pa
    f, _ = pa.pa_rope_frequencies(rotary, base)
    rng = np.random.default_rng(int(base))
    pos = [0, 1, 131071, 2 ** 31, 2 ** 40 + 1, -(2 ** 45) - 7, *(int(x) for x in rng.integers(2 ** 49, 2 ** 50, 60))]
    t = len(pos)
    x = torch.zeros(t, 1, rotary, device="cuda")
    x[..., :rotary // 2] = 1.0                       # (cos, sin) of every pair
    out, k_out = torch.empty_like(x), torch.empty_like(x)
    pa.pa_rope(out, k_out, x, x, torch.tensor(pos, device="cuda"), f.cuda())
    got = out.double().cpu().numpy()[:, 0]
    inv = inverse_two_pi()
    exact = np.array([[turns(p, fi, inv) for fi in f.tolist()] for p in pos]) * 2 * np.pi
    slack = np.abs(np.array(pos, float))[:, None] * 2.0 ** -65 * 2 * np.pi * (1 + 2.0 ** -6) + 2.0 ** -22
    for part, ref in ((got[:, :rotary // 2], np.cos(exact)), (got[:, rotary // 2:rotary], np.sin(exact))):
        worst = np.max(np.abs(part - ref) / slack)
        assert worst <= 1.0, f"{worst:.2f} times the bound"

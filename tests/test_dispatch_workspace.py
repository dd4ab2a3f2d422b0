"""The dispatch plan's workspace: one of the largest sizes serves every smaller call (no GPU is needed)."""
import itertools
import random

import pytest

import __graft_entry__

__graft_entry__.build()
import trellis_quantized_moe_gb300 as X  # noqa: E402
from trellis_quantized_moe_gb300 import binding as B  # noqa: E402

P = 1 << 20          # an aligned address that nothing dereferences
EXPERTS = [1, 2, 7, 8, 64, 192, 256, 288, 510, 511, 512, 513, 600, 1000, 1023, 1024]
ROUTES = [0, 1, 512, 8192, 32767, 32768, 32769, 33793, 40000, 63488, 64513, 65536, 131071, 131072, 131073, 1 << 20, (1 << 30) - 1]


def needed(R, E):
    """Bytes that the kernels use: 64 words, and E + 2 counts of every CTA where these are no cluster."""
    ctas = 0 if R <= 32768 else min(-(-R // 1024), 128, 65536 // (E + 1))
    return 4 * (64 + ctas * (E + 2))


def test_bytes_never_fall_and_are_enough():
    size = {(R, E): X.exl3_dispatch_workspace_bytes(R, 1, E) for R in ROUTES for E in EXPERTS}
    for (R, E), n in size.items():
        assert n >= needed(R, E) and n % 256 == 0
    for (r0, r1), (e0, e1) in itertools.product(zip(ROUTES, ROUTES[1:]), zip(EXPERTS, EXPERTS[1:])):
        assert size[r0, e0] <= size[r0, e1] and size[r0, e0] <= size[r1, e0]


def test_bytes_never_fall_for_drawn_sizes():
    rng = random.Random(5)
    for _ in range(20000):
        M, k, E = int(2 ** rng.uniform(0, 24)), rng.randint(1, 32), rng.randint(1, 1024)
        M1, k1, E1 = rng.randint(0, M), rng.randint(1, k), rng.randint(1, E)
        n = X.exl3_dispatch_workspace_bytes(M, k, E)
        assert X.exl3_dispatch_workspace_bytes(M1, k1, E1) <= n and needed(M * k, E) <= n


@pytest.mark.parametrize("M,k,E", [(1 << 17, 8, 511), (5000, 8, 1024), (100, 8, 192)])
def test_a_smaller_workspace_is_refused(M, k, E):
    n = X.exl3_dispatch_workspace_bytes(M, k, E)
    call = lambda b: B.lib().exl3_dispatch_plan(P, 3, M, k, E, P, P, P, P, P, b, None)
    assert call(n - 1) == -6

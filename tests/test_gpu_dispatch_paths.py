"""The dispatch plan's every path with ids that are bad, missing or all the same.

A case says which path it is for and checks that it takes it: the counts that CTAs by
themselves leave are all that a workspace holds beyond its first 256 bytes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import trellis_quantized_moe_gb300 as X  # noqa: E402
from test_gpu_dispatch import Plan, check_plan, make_ids  # noqa: E402

E = 97
# one CTA, clusters of both thread counts, counted CTAs, counted CTAs whose warps walk more steps than registers hold
PATHS = {"cta": (60, 8), "cluster": (1500, 4), "wide cluster": (7000, 4), "counted": (9000, 4), "parked": (140000, 4)}


def path_of(R):
    counts = (X.exl3_dispatch_workspace_bytes(R, 1, E) - 256) // (4 * (E + 2))
    if counts == 0:
        return "cta" if R <= 512 else "cluster" if R <= 8192 else "wide cluster"
    return "parked" if R > counts * 1024 * 4 else "counted"


@pytest.fixture(params=PATHS)
def sizes(request):
    M, k = PATHS[request.param]
    assert path_of(M * k) == request.param
    return M, k


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("where", ["first", "middle", "last", "nowhere"])
@pytest.mark.parametrize("bad", [E, -2])
def test_a_bad_id_anywhere(sizes, dtype, where, bad):
    M, k = sizes
    ids = make_ids(M, E, k, M, 0.1, dtype=dtype)
    at = {"first": 0, "middle": M * k // 2 + 1, "last": M * k - 1}
    if where in at:
        ids.view(-1)[at[where]] = bad if dtype is torch.int32 else bad * (1 << 33)
    p = Plan(ids, E)
    assert X.exl3_workspace_error(p.ws) == (1 if where in at else 0)
    check_plan(p, ids, E)


def test_every_id_bad(sizes):
    M, k = sizes
    ids = torch.full((M, k), -5, dtype=torch.int32, device="cuda")
    p = Plan(ids, E)
    assert X.exl3_workspace_error(p.ws) == 1
    check_plan(p, torch.full_like(ids, -1), E)


def test_one_expert_none_and_repeats(sizes):
    M, k = sizes
    for ids in (torch.full((M, k), E - 1), torch.full((M, k), -1), torch.zeros((M, k)),
                torch.arange(M * k).reshape(M, k) % 3, torch.arange(M * k).reshape(M, k) % (E + 1) - 1):
        ids = ids.to(torch.int32).cuda()
        p = Plan(ids, E)
        assert X.exl3_workspace_error(p.ws) == 0
        check_plan(p, ids, E)


def test_the_error_word_is_the_calls_own(sizes):
    """A good batch after a bad one in the same workspace, and the other way round."""
    M, k = sizes
    ids = make_ids(M, E, k, 3)
    p = Plan(ids, E)
    for bad in (True, False, True):
        ids[M - 1, k - 1] = E if bad else 5
        p.go()
        assert X.exl3_workspace_error(p.ws) == int(bad)
        check_plan(p, ids, E)


@pytest.mark.parametrize("experts", [8, 200, 511, 1000])
def test_a_workspace_of_the_largest_serves_smaller_batches(experts):
    """Its contents are of calls of other sizes; nothing behind the bytes of the call's own sizes is needed."""
    ws = torch.randint(0, 255, (X.exl3_dispatch_workspace_bytes(140000, 4, 1024),), dtype=torch.uint8, device="cuda")
    for M, k in list(PATHS.values()) + list(PATHS.values())[::-1]:
        ids = make_ids(M, experts, k, M, 0.1)
        p = Plan(ids, experts)
        for t in (p.offsets, p.packed, p.slots, p.experts):
            t.fill_(-77)
        X.exl3_dispatch_plan(ids, experts, p.offsets, p.packed, p.slots, ws, experts=p.experts)
        assert X.exl3_workspace_error(ws) == 0
        check_plan(p, ids, experts)

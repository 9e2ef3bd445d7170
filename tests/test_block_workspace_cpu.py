"""Size of the router gradient's workspace: at least what the worst grouping needs, at most about one partial
row per unit of routes and expert."""
import pytest

from sparse_moe_routed_gb300 import moe_route_backward_workspace_size as size


def unit(R):
    """Routes per unit, as route_grad.cu cuts them."""
    return 64 if R <= 16000 else 128 if R <= 100000 else 256


@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (520, 1, 8, 64), (4096, 10, 512, 2560), (1 << 20, 8, 64, 2560),
                                     (1 << 23, 1, 1024, 128), (1 << 20, 32, 32, 4096), (100, 1, 1024, 8)])
def test_router_gradient_workspace(T, k, E, H):
    R = T * k
    u = unit(R)
    # most partial rows: as many experts as there are with one route more than a unit, the rest in whole units
    several = min(E, R // (u + 1))
    worst = 2 * several + (R - several * (u + 1)) // u
    units, multi = E + R // u, min(E, R // u)
    rows = R // u + multi + 1
    assert worst <= rows
    tables = 16 * units + 16 * multi + 4 * rows
    got = size(T, k, E, H)
    assert 4 * worst * H <= got <= 4 * rows * H + tables + 4 * 256

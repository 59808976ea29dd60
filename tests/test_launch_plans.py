"""The launches of the residual norms' gradient, on the host."""
import launch_record as lr

FAKE = 0x10000   # 16-byte aligned, never dereferenced
TYPES = "qqpiqpqpiqpiqipppiqqddipipppppqpqpppppp" + "zp"


def grad(rows, cols, gate_rows=0, bf16=1, post=1):
    """Arguments of fp4q_residual_norm_grad with everything asked for."""
    gate, vec = (FAKE if gate_rows else 0), (FAKE if post != 2 else 0)
    return ("fp4q_residual_norm_grad", TYPES,
            [rows, cols, FAKE, bf16, cols, FAKE, cols, FAKE, bf16, cols, FAKE, bf16, cols, post, vec, vec, gate, 0,
             gate_rows, cols, 1.0, 1.0, 1, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, cols, FAKE, cols, vec, vec, gate,
             FAKE, FAKE, FAKE, 1 << 50, 0])


def test_a_launch_holds_below_2_to_32_threads_a_side(tmp_path):
    """Rows of up to 2^31 - 1 columns, any number of gates: every column is
    joined, and no launch is larger than a launch can be."""
    sizes = [(2, c, g) for c in ((1 << 28) - 64, 1 << 28, (1 << 28) + 40, (1 << 31) - 1) for g in (0, 1)]
    sizes += [((1 << 31) - 1, 64, g) for g in (0, 1, 1000)] + [(1, 1, 0), (70000, 8192, 300), (300, 20000, 7)]
    for (rows, cols, g), (status, seen) in zip(sizes, lr.launches(tmp_path, [grad(*s) for s in sizes])):
        assert status == 0
        for kernel, _, (x, y, z), threads in seen:
            assert x * threads < 1 << 32 and y < 1 << 16 and z == 1, (rows, cols, g, kernel, x, y, threads)
        joins = [grid[0] for kernel, _, grid, _ in seen if kernel == "residual_grad_join_kernel"]
        assert not joins or sum(joins) == -(-cols // 64)


def test_teams_of_waves_have_rows(tmp_path):
    """Gates of any length: slabs of whole groups fit on the card together, and
    where half of the teams would have no group, the walk is short."""
    sizes = [(R, C, g) for R in (4096, 16384, 49152) for C in (256, 512, 600, 1024, 1500, 2048, 5120)
             for g in (1, 2, 5, 8, 12, 16, 21, 24, 31, 32, 40, 48, 63, 64, 65, 96, 100, 128, 160, 192)]
    whole = 0
    for (R, C, g), (status, seen) in zip(sizes, lr.launches(tmp_path, [grad(*s) for s in sizes])):
        assert status == 0
        kernel, (_, _, _, gate, T, _), (count, _, _), threads = seen[0]
        assert kernel == "residual_grad_kernel"
        if not gate:
            continue
        whole += 1
        teams = threads // 64 // (-(-C // 512) if T else 1)
        groups = -(-R // g)                        # of all rows
        each = -(-groups // count)                 # of a slab, about
        turns = -(-each // teams)
        assert count <= 256 * max(1, 512 // threads), (R, C, g, count)
        assert 2 * each > turns * teams or turns * g <= 16, (R, C, g, count, teams)
    assert 0 < whole < len(sizes)

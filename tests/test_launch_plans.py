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

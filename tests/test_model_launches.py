"""The launches of the model operators at their largest sizes, without a GPU.

HIP takes no launch whose grid has 2^32 or more work-items along a dimension, and
at most 65535 workgroups along the second and third.  A child process preloads a library that
stands in for hipLaunchKernel: it writes down every launch and runs none, so that the
C ABI's host code can be driven with sizes and addresses that no card holds."""
import ctypes
import os
import subprocess
import sys
import textwrap

import pytest

import gated_convolution_sequence_amd as hc
from gated_convolution_sequence_amd.model import _Tensor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = textwrap.dedent('''
    #include <cstddef>
    #include <cstdint>
    #include <cstdio>
    #include <cstdlib>
    // the types of the runtime's header by size: dim3 is three 32-bit words, an error an int.  A launch pushes
    // its grid and block, and the kernel's stub takes them off again.
    struct dim3 { uint32_t x, y, z; };
    static dim3 the_grid, the_block;
    extern "C" {
    int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, void *) {
        the_grid = grid, the_block = block;
        return 0;
    }
    int __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, void **stream) {
        *grid = the_grid, *block = the_block, *lds = 0, *stream = nullptr;
        return 0;
    }
    int hipLaunchKernel(const void *, dim3 grid, dim3 block, void **, size_t, void *) {
        FILE *f = fopen(getenv("LAUNCH_LOG"), "a");
        fprintf(f, "%u %u %u %u %u %u\\n", grid.x, grid.y, grid.z, block.x, block.y, block.z);
        fclose(f);
        return 0;
    }
    int hipGetLastError(void) { return 0; }
    }
''')

CHILD = textwrap.dedent('''
    import sys
    sys.path.insert(0, sys.argv[1]); sys.path.insert(0, sys.argv[1] + "/tests")
    import gated_convolution_sequence_amd as hc
    import test_model_launches as cases
    L = hc.model_lib()
    for name in sys.argv[2:]:
        with open(cases.os.environ["LAUNCH_LOG"], "a") as f:
            f.write("case %s\\n" % name)
        st = cases.CASES[name](L)
        assert st == (-7 if "refused" in name else 0), (name, st, hc.model_strerror(st))
''')


def P(i):
    """An address far from the others."""
    return (1 << 55) + (i << 50)


HUGE = 1 << 49  # bytes of a workspace that no size here outgrows


def xent_fwd(M, K, V, dtype, ldx=None):
    return lambda L: L.hyena_xent_fwd(P(0), P(1), None, P(2), M, K, V, ldx or K, P(3), P(4), P(5), HUGE, dtype, None)


def xent_bwd(M, K, V, dtype, dx=True, dw=True, db=True):
    return lambda L: L.hyena_xent_bwd(P(0), P(1), P(2), P(3), P(4), P(5), M, K, V, K, K, P(6) if dx else None,
                                      P(7) if dw else None, P(8) if db else None, P(9), HUGE, dtype, None)


def norm_fwd(M, D, dtype):
    return lambda L: L.hyena_norm_fwd(P(0), P(1), P(2), M, D, D, D, 0, 1e-5, P(3), P(4), P(5), dtype, None)


def norm_bwd(M, D, dtype, dx=True):
    return lambda L: L.hyena_norm_bwd(P(0), P(1), P(2), P(3), P(4), M, D, D, D, D, 0, P(5) if dx else None, P(6), P(7), P(8),
                                      HUGE, dtype, None)


def table(sizes):
    """A list of tensors, their arrays 2^43 bytes apart."""
    t = (_Tensor * len(sizes))()
    for k, (e, n) in enumerate(zip(t, sizes)):
        at = [(1 << 54) + ((7 * k + j) << 43) for j in range(7)]
        e.param, e.grad, e.exp_avg, e.exp_avg_sq, e.exp_avg_scale, e.exp_avg_sq_scale, e.master = at
        e.numel = n
    return t


def adamw(sizes, bits, dtype=0):
    def call(L, t=table(sizes)):
        return L.hyena_adamw_step(ctypes.addressof(t), len(t), 1e-3, 0.9, 0.95, 1e-8, 0.1, 1, 0, None, None, None, None, bits,
                                  dtype, None)
    return call


def grad_norm(sizes, dtype=0):
    def call(L, t=table(sizes)):
        return L.hyena_grad_norm(ctypes.addressof(t), len(t), 1.0, P(9), P(10), P(11), HUGE, dtype, None)
    return call


# elements: 2048 a workgroup with moments of 8 bits, 4096 of 32 bits, 32768 for the norm
LISTS = {
    "adamw8 2^24": ([1 << 31] * 16, 2048), "adamw8 past": ([5, (1 << 31) + 77, 0] * 30, 2048),
    "adamw8 one": ([(1 << 40) - 1], 2048), "adamw8 ones": ([(1 << 40) - 1] * 5, 2048),
    "adamw32 2^24": ([1 << 33] * 8, 4096), "adamw32 one": ([(1 << 40) - 1] * 2, 4096),
    "adamw32 many": ([(1 << 36) + 1, 9] * 70, 4096),
    "norm 2^24": ([1 << 36] * 8, 32768), "norm many": ([(1 << 40) - 1] * 100, 32768), "norm small": ([3] * 100, 32768),
}


MOST = (1 << 31) - 1024  # rows, entries
BF16, F32 = 0, 1
CASES = {
    # logits from 2^36 on in 64 x 64 tiles of fp32, from 2^38 and 2^39 in those of bf16
    "fwd f32 2^36": xent_fwd(1 << 20, 64, 1 << 16, F32),
    "fwd f32 2^36 odd": xent_fwd((1 << 20) + 1, 7, (1 << 16) + 1, F32),
    "fwd f32 past": xent_fwd(1 << 22, 16, 1 << 17, F32),
    "fwd bf16 2^38": xent_fwd(1 << 22, 8, 1 << 16, BF16),
    "fwd bf16 2^39 odd": xent_fwd((1 << 22) - 1, 7, 1 << 17, BF16),
    "fwd bf16 many": xent_fwd(1 << 24, 64, 1 << 18, BF16),
    # most rows, most entries
    "fwd rows f32": xent_fwd(MOST, 1, 2, F32), "fwd rows bf16": xent_fwd(MOST, 8, 2, BF16),
    "fwd rows / 2": xent_fwd(1 << 30, 1, 3, F32), "fwd rows / 4": xent_fwd(1 << 29, 1, 3, BF16),
    "fwd few rows": xent_fwd(16, 8, MOST, BF16), "fwd few rows f32": xent_fwd(1, 1, 1 << 27, F32),
    "fwd few tiles": xent_fwd(17, 8, MOST, BF16), "fwd few tiles f32": xent_fwd(64, 3, MOST, F32),
    "bwd rows f32": xent_bwd(MOST, 1, 2, F32), "bwd rows bf16": xent_bwd(MOST, 8, 2, BF16),
    "bwd rows / 2": xent_bwd(1 << 30, 1, 3, F32), "bwd rows wide": xent_bwd(1 << 28, 256, 256, F32),
    "bwd rows dx": xent_bwd(1 << 28, 1024, 128, BF16, dw=False, db=False),
    "bwd pieces": xent_bwd(1 << 25, 8, 2048, F32), "bwd entries": xent_bwd(4, 8, 1 << 27, BF16),
    "bwd entries f32": xent_bwd(70, 5, 1 << 26, F32),
    # more tiles than 31 bits number: said before the first launch
    "fwd refused f32": xent_fwd(1 << 22, 8, 1 << 21, F32), "fwd refused bf16": xent_fwd(1 << 23, 8, 1 << 22, BF16),
    "bwd refused": xent_bwd(1 << 30, 1 << 17, 2, BF16), "bwd refused w": xent_bwd(2, 1 << 17, 1 << 30, BF16),
    "fwd largest": xent_fwd(1 << 22, 8, 1 << 20, F32), "bwd largest": xent_bwd(1 << 22, 8, 1 << 20, F32),
    # rows of all lengths; dw and db of 2^28 and more channels
    "rows fwd": norm_fwd(3, 1 << 31, BF16), "rows fwd many": norm_fwd(1 << 40, 16, F32),
    "rows bwd 2^28": norm_bwd(1, 1 << 28, BF16), "rows bwd f32": norm_bwd(300, (1 << 28) + 3, F32),
    "rows bwd most": norm_bwd(2, 1 << 31, F32), "rows bwd dw": norm_bwd(2, 1 << 31, BF16, dx=False),
    "rows bwd many": norm_bwd(1 << 40, 16, BF16),
    **{name: grad_norm(sizes) if name.startswith("norm") else adamw(sizes, 8 if "8" in name.split()[0] else 32)
       for name, (sizes, _) in LISTS.items()},
}


def launches(tmp_path, names):
    """[(grid, block)] of each case."""
    lib, log, source = (str(tmp_path / n) for n in ("stub.so", "launches", "stub.cpp"))
    with open(source, "w") as f:
        f.write(STUB)
    subprocess.run(["g++", "-shared", "-fPIC", "-o", lib, source], check=True)
    first = " ".join(filter(None, (lib, os.environ.get("LD_PRELOAD"))))  # before what is preloaded already
    env = dict(os.environ, LD_PRELOAD=first, LAUNCH_LOG=log)
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, *names], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    out = {}
    for line in open(log):
        if line.startswith("case "):
            rows = out.setdefault(line[5:].rstrip(), [])
        else:
            v = list(map(int, line.split()))
            rows.append((v[:3], v[3:]))
    return out


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(hc.MODEL_LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()


def check_launches(tmp_path, names):
    found = launches(tmp_path, names)
    assert sorted(found) == sorted(names)
    for name, rows in found.items():
        assert bool(rows) == ("refused" not in name), name
        for grid, block in rows:
            assert all(g * b < 1 << 32 for g, b in zip(grid, block)), (name, grid, block)
            assert max(grid[1:]) < 1 << 16 and min(grid) >= 1 and block[0] * block[1] * block[2] <= 1024, (name, grid, block)
    return found


def test_readout_launches(tmp_path):
    found = check_launches(tmp_path, [n for n in CASES if n.split()[0] in ("fwd", "bwd")])
    # enough workgroups for the logits' tiles (for the merging of 32 rows each), and less than a row of 2^21 more
    for name, tiles in (("fwd f32 2^36", 1 << 24), ("fwd f32 2^36 odd", ((1 << 14) + 1) * ((1 << 10) + 1)),
                        ("fwd rows f32", MOST // 32), ("fwd few rows", MOST // 16), ("fwd largest", 1 << 30)):
        most = max(grid[0] * grid[1] for grid, _ in found[name])
        assert tiles <= most < tiles + (1 << 21), (name, most)


def test_launches_over_lists_of_tensors(tmp_path):
    """Every tensor's workgroups are launched, 48 tensors or 2^30 workgroups at a time."""
    found = check_launches(tmp_path, list(LISTS))
    for name, (sizes, span) in LISTS.items():
        rows = found[name][:-1] if name.startswith("norm") else found[name]  # the last one adds up the norm
        want = sum(-(-n // span) for n in sizes)
        got = [grid[0] * grid[1] for grid, _ in rows]
        # (a launch of more than 2^21 is filled up to whole rows of that many)
        assert want <= sum(got) < want + len(got) * (1 << 21) and max(got) <= 1 << 30, (name, want, got)
        assert len(got) >= -(-sum(n > 0 for n in sizes) // 48)


def test_norm_launches(tmp_path):
    found = check_launches(tmp_path, [n for n in CASES if n.startswith("rows")])
    for name, D in (("rows bwd 2^28", 1 << 28), ("rows bwd f32", (1 << 28) + 3), ("rows bwd most", 1 << 31)):
        grid, _ = found[name][-1]  # 64 columns a workgroup, for dw and for db
        assert -(-D // 64) <= grid[0] * grid[1] < -(-D // 64) + (1 << 21) and grid[2] == 2, (name, grid)

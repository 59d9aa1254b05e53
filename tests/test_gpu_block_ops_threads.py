"""Calls of the operators around a projection from several host threads at once."""
import ctypes
import subprocess
import threading

import pytest
import torch

from gpu_common import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    return require_cuda()


LOOP = """
typedef int (*entry)(const void *, void *);
int refused(entry f, const void *args, void *stream, int n) {
    int bad = 0;
    for (int i = 0; i < n; ++i) bad += f(args, stream) != 0;
    return bad;
}
"""


@pytest.fixture(scope="module")
def loop(tmp_path_factory):
    """Calls an entry point n times without Python (and its lock) in between."""
    d = tmp_path_factory.mktemp("loop")
    (d / "loop.c").write_text(LOOP)
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-o", str(d / "loop.so"), str(d / "loop.c")], check=True)
    f = ctypes.CDLL(str(d / "loop.so")).refused
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int]
    return f


@pytest.mark.parametrize("widths", [(8192, 512), (4096, 8192), (8192, 2048, 4096, 512)])
def test_norms_of_other_widths_at_once(nv, loop, widths):
    """Each thread its own rows on its own stream: none is refused, whatever
    shared memory the others' widths take."""
    entry = ctypes.cast(nv.lib().nvfp4_residual_norm, ctypes.c_void_p)
    start, bad, calls = threading.Barrier(len(widths)), [], []
    for cols in widths:
        rows = (1 << 21) // cols + 1
        x = torch.randn(rows, cols, device="cuda").to(torch.bfloat16)
        out = torch.empty_like(x)
        args = nv.ResidualNormArgs(rows=rows, cols=cols, residual=x.data_ptr(), residual_stride=cols,
                                   out=out.data_ptr(), out_stride=cols, groups=1, residual_scale=1.0,
                                   branch_scale=1.0, pre_norm=1, pre_eps=1e-6)
        calls.append((args, x, out, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def run(args, x, out, stream):
        start.wait()
        bad.append(loop(entry, ctypes.addressof(args), stream.cuda_stream, 4000))

    threads = [threading.Thread(target=run, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert bad == [0] * len(widths)
    for _, x, out, _ in calls:
        assert torch.equal(out, nv.residual_norm(x, pre=nv.Norm()).out)

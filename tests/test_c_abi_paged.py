"""The paged-cache calls used from plain C (tests/c_abi/paged.c): compiled with
gcc against the header alone on the CPU; on the GPU its outputs must equal, bit
for bit, what the Python binding returns for the same inputs."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from block_sparse_long_score_b200 import build as xbuild
from block_sparse_long_score_b200 import xattn as X

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = "/usr/local/cuda"


def _compile(tmp_path):
    xbuild.build()
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    exe = str(tmp_path / "paged")
    libdir = os.path.dirname(X.library_path())
    cmd = [gcc, "-std=c11", "-O1", "-Wall", "-Wextra", "-Werror",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(CUDA, "include"),
           os.path.join(ROOT, "tests", "c_abi", "paged.c"), "-o", exe,
           "-L", libdir, "-lxattn", "-L", os.path.join(CUDA, "lib64"), "-lcudart",
           f"-Wl,-rpath,{libdir}", f"-Wl,-rpath,{os.path.join(CUDA, 'lib64')}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def test_c_program_compiles_against_the_header_alone(tmp_path):
    assert os.path.exists(_compile(tmp_path))


@pytest.mark.gpu
def test_c_program_matches_the_binding(tmp_path):
    from block_sparse_long_score_b200 import (xattn_paged_append, xattn_paged_decode,
                                              xattn_paged_plan)
    exe = _compile(tmp_path)
    fresh, hq, hkv, d, page, pages, rows = [70, 0, 16, 1, 333], 8, 2, 128, 16, 40, 24
    n, T = len(fresh), sum(fresh)
    g = torch.Generator().manual_seed(1)
    Q, K, V = (torch.randn(*s, generator=g).to(torch.bfloat16)
               for s in ((n, hq, d), (T, hkv, d), (T, hkv, d)))
    inp, out = tmp_path / "in.bin", tmp_path / "out.bin"
    inp.write_bytes(b"".join(t.view(torch.int16).numpy().tobytes() for t in (Q, K, V)))
    args = [exe, str(inp), str(out)] + [str(x) for x in (n, hq, hkv, d, page, pages, rows, *fresh)]
    r = subprocess.run(args, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)
    raw = out.read_bytes()
    O = torch.from_numpy(np.frombuffer(raw[:Q.numel() * 2], dtype=np.int16).copy())
    lse = torch.from_numpy(np.frombuffer(raw[Q.numel() * 2:-4 * T], dtype=np.float32).copy())
    slots = torch.from_numpy(np.frombuffer(raw[-4 * T:], dtype=np.int32).copy())

    i32 = dict(dtype=torch.int32, device="cuda:0")
    kp, vp = (torch.zeros(pages, hkv, page, d, dtype=torch.bfloat16, device="cuda:0")
              for _ in range(2))
    table = torch.zeros(n, rows, **i32)
    lens, _, _, sl = xattn_paged_plan(
        torch.zeros(n, **i32), torch.tensor(fresh, **i32), torch.tensor([0, pages], **i32),
        torch.arange(pages - 1, -1, -1, **i32), table, page, max_tokens=T)
    xattn_paged_append(K.cuda(), V.cuda(), sl, kp, vp)
    want, want_lse = xattn_paged_decode(Q.cuda(), kp, vp, table, lens, lse=True)
    torch.cuda.synchronize()
    assert torch.equal(slots, sl.cpu())
    assert torch.equal(O.view(torch.bfloat16).reshape(Q.shape), want.cpu())
    assert torch.equal(lse.reshape(n, hq), want_lse.cpu())

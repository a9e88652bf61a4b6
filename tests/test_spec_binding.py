"""The compiled binding of the speculative calls with tensors that have no
storage: an exception, not the end of the process."""
import subprocess
import sys

import pytest
import torch

import paged_kv_cache_mapping_gb300 as pkv
from paged_kv_cache_mapping_gb300 import build as pkv_build
from tests.conftest import ROOT

HEAD = """
import torch, paged_kv_cache_mapping_gb300 as pkv
from torch._subclasses.fake_tensor import FakeTensorMode
def refused(call):
    try:
        call()
    except (RuntimeError, NotImplementedError, pkv.PkvError) as e:
        print("refused", type(e).__name__)
    else:
        raise SystemExit("accepted")
sparse = lambda: torch.sparse_coo_tensor(torch.zeros(1, 1, dtype=torch.long, device="cuda"),
                                         torch.zeros(1, dtype=torch.int32, device="cuda"), (2,))
with FakeTensorMode():  # CUDA tensors without a GPU
    i = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
"""
BODIES = {
    "vmap mask": "    refused(lambda: torch.vmap(lambda a: pkv.pkv_tree_mask(a, a, a, 1))(i))",
    "vmap commit": "    refused(lambda: torch.vmap(lambda a: pkv.pkv_tree_commit(a, a, a, a, a, a, a, a))(i))",
    "vmap attention": "    refused(lambda: torch.vmap(lambda a: pkv.pkv_tree_attention(a, a, a, a, a, a, a, 1.0, a, workspace=a))(i))",
    "vmap rope": "    refused(lambda: torch.vmap(lambda a: pkv.pkv_rope_append(a, a, a, a, a, pkv.pkv_rope_init(2), a, a, a))(i))",
    "sparse commit": "    refused(lambda: pkv.pkv_tree_commit(*[sparse()] * 8))",
    "sparse mask": "    refused(lambda: pkv.pkv_tree_mask(i[0], i[0], i[0], 1, sparse(), i[0]))",
    "sparse workspace": "    refused(lambda: pkv.pkv_tree_attention(*[i] * 7, 1.0, i, workspace=sparse()))",
}


@pytest.mark.parametrize("name", list(BODIES))
def test_tensors_without_storage_are_refused(name):
    pkv_build.build()
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", HEAD + BODIES[name]], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.startswith("refused"), (r.returncode, r.stderr[-2000:])


@pytest.mark.gpu
def test_tensors_without_storage_are_refused_on_the_gpu():
    i = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    sparse = torch.zeros(2, dtype=torch.int32, device="cuda").to_sparse()
    for call in (lambda: torch.vmap(lambda a: pkv.pkv_tree_mask(a, a, a, 1))(i),
                 lambda: pkv.pkv_tree_commit(*[sparse] * 8),
                 lambda: pkv.pkv_tree_mask(i[0], i[0], i[0], 1, sparse, i[0])):
        with pytest.raises((RuntimeError, pkv.PkvError)):
            call()
    # and the next call works
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    mask, pos = pkv.pkv_tree_mask(one - 1, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), one + 5, 1)
    assert mask.tolist() == [[1]] and pos.tolist() == [4]
    assert pkv.pkv_device_errors() == 0

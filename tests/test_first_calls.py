"""First calls of a process that come from several host threads at once."""
import os
import shutil
import subprocess
import sys

import pytest

from masked_attention_backward_gb300 import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# The driver's entry point is looked up by a stand-in that takes its time.
LOOKUP = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
#include "tmap.h"

static std::atomic<int> lookups{0};
static CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                       const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                       CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                       CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
extern "C" cudaError_t CUDARTAPI cudaGetDriverEntryPointByVersion(
    const char*, void** fn, unsigned int, unsigned long long,
    cudaDriverEntryPointQueryResult* found) {
  ++lookups;
  std::this_thread::sleep_for(std::chrono::milliseconds(300));
  *fn = reinterpret_cast<void*>(&encode);
  *found = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

int main() {
  constexpr int N = 8;
  std::atomic<int> ready{0}, failed{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < N; ++i)
    threads.emplace_back([&] {
      ++ready;
      while (ready < N) std::this_thread::yield();
      if (!mab::get_encode_tiled()) ++failed;
    });
  for (auto& t : threads) t.join();
  std::printf("%d lookups, %d of %d threads got nothing\n", lookups.load(), failed.load(), N);
  return failed == 0 && lookups == 1 ? 0 : 1;
}
"""


def test_the_tensor_map_encoder_is_found_by_every_thread(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "lookup.cpp", tmp_path / "lookup"
    src.write_text(LOOKUP)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(b.nvcc()))), "include")
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", b.CSRC, "-I", cuda, str(src), "-o",
                    str(exe)], check=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr


CALLS = r"""
import math, threading
import torch
from masked_attention_backward_gb300 import binding as mab

N = 6
q = torch.randn(1, 2, 64, 128, device="cuda").half()
pages = torch.randn(4, 2, 16, 128, device="cuda").half()
cache = mab.PagedCache(pages, pages)
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
table, qp = i32([[0, 1, 2, 3]]), q[0].transpose(0, 1).contiguous()
mask = mab.Mask(kind=mab.ATTN_MASK_CAUSAL, cu_seqlens_q=i32([0, 64]), seqlen_k=i32([64]),
                total_q=64, max_seqlen_q=64, max_seqlen_k=64)
calls = [lambda: mab.paged_fwd(qp, cache, table, None, mask, 0.1),
         lambda: mab.fwd(q, q, q, None, mab.Mask(kind=mab.ATTN_MASK_CAUSAL), 0.1)]
mab.load()
torch.cuda.synchronize()
gate, errors = threading.Barrier(N), []

def go(i):
    with torch.cuda.stream(torch.cuda.Stream()):
        gate.wait()
        try:
            calls[i % 2]()
        except Exception as e:
            errors.append(e)

threads = [threading.Thread(target=go, args=(i,)) for i in range(N)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not errors, errors
"""


@pytest.mark.gpu
def test_first_calls_of_a_process_from_several_threads(cuda_lib):
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", CALLS], cwd=ROOT, capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr

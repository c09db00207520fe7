"""How the prompts' attention ends, from its source (a wait that runs out cannot be brought about without a hang)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tensor_memory_is_freed_behind_a_commit_of_all_mmas():
    """One barrier is committed once, behind the issuing loop, whatever made it end; the issuing warp waits for that
    phase alone, all warps meet, and only then is the tensor memory freed. (A phase that a step's MMAs complete too
    may have passed long before the last of them.)"""
    src = open(os.path.join(ROOT, "gemm_gguf_block_gb300", "csrc", "attn_tiles.cu")).read()
    src = re.sub(r"//[^\n]*", "", src)
    commit = [m.start() for m in re.finditer(r"commit_lead\(&bars\[B_DRAINED\]", src)]
    wait = [m.start() for m in re.finditer(r"wait_or_abort_sleep\(&bars\[B_DRAINED\], 0,", src)]
    assert len(commit) == len(wait) == 1 and len(re.findall(r"mbar_init\(&bars\[B_DRAINED\], 1\)", src)) == 1
    last_mma = max(m.end() for m in re.finditer(r"\b(?:scores|product)\(", src))
    free = [m.start() for m in re.finditer(r"tmem_dealloc\(", src)]
    assert last_mma < commit[0] < wait[0] < free[0] and len(free) == 1
    assert "__syncthreads()" in src[wait[0]:free[0]]
    assert "break" not in src[commit[0]:free[0]] and "return" not in src[commit[0]:free[0]]
    numbers = re.search(r"enum \{([^}]*B_DRAINED[^}]*)\}", src).group(1)
    first = {k: int(v) for k, v in re.findall(r"(B_\w+) = (\d+)", numbers)}
    assert first["B_DRAINED"] >= first["B_FREE"] + 2 and (first["B_DRAINED"] + 1) * 8 <= 1024

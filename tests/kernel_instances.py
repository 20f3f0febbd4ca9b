"""Which kernel instances the library holds, and which a call launches."""
import re
import shutil
import subprocess

import torch

import expert_weight_residency_amd as moe


def instances(text, names):
    """name<arguments> of the template kernels whose names match the pattern."""
    return set(re.findall(rf"\b((?:{names})<[^>]*>)\(", text.replace("__device_stub__", "")))


def held(names):
    nm = shutil.which("nm")
    assert nm, "nm lists the library's kernels"
    return instances(subprocess.run([nm, "-C", moe.LIB_PATH], capture_output=True, text=True,
                                    check=True).stdout, names)


def launched(f, names):
    """The instances that f launches (once more if the profiler delivered no
    event at all)."""
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    for _ in range(3):
        with profile(activities=[ProfilerActivity.CUDA], acc_events=True) as p:
            f()
            torch.cuda.synchronize()
        got = instances("\n".join(e.key for e in p.key_averages()), names)
        if got:
            break
    return got

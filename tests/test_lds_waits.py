"""Muon's products fetch from memory straight into LDS, and past the last stage they fetch again what nobody reads.  Their epilogue writes
to the same LDS, so each wave has to wait for its own fetches before the barrier between the two.  Read from the assembly of this
library's own build."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "all_gather_amd", "csrc")
LLVM = "/opt/rocm/llvm/bin"

pytestmark = pytest.mark.skipif(not os.path.exists(f"{LLVM}/llvm-objdump"), reason="ROCm toolchain not present")


def assembly(src, tmp):
    """Lines of each kernel of a source file: from the library's object where that is newer than the file, else compiled here."""
    from all_gather_amd import _build

    obj = os.path.join(_build.OBJ, os.path.splitext(src)[0] + ".o")
    files = [os.path.join(CSRC, f) for f in (src, "mr_train.h", "packs.h")]
    if not os.path.exists(obj) or os.path.getmtime(obj) < max(map(os.path.getmtime, files)):
        obj = str(tmp / "kernels.o")
        r = subprocess.run([_build.hipcc(), *_build.CFLAGS, "-c", files[0], "-o", obj], capture_output=True, text=True, timeout=900)
        assert r.returncode == 0, r.stderr[-2000:]
    fat, co = str(tmp / "fat.bin"), str(tmp / "kernels.co")
    for cmd in ([f"{LLVM}/llvm-objcopy", f"--dump-section=.hip_fatbin={fat}", obj, str(tmp / "host.o")],
                [f"{LLVM}/clang-offload-bundler", "--unbundle", "--type=o", f"--input={fat}", "--targets=hipv4-amdgcn-amd-amdhsa--gfx950",
                 f"--output={co}"]):
        subprocess.run(cmd, check=True, capture_output=True, timeout=300)
    text = subprocess.run([f"{LLVM}/llvm-objdump", "-d", co], check=True, capture_output=True, text=True, timeout=300).stdout
    out, name = {}, None
    for line in text.splitlines():
        m = re.match(r"[0-9a-f]+ <(\S+)>:", line)
        if m:
            name = m.group(1)
            out[name] = []
        elif name and line.startswith("\t"):
            out[name].append(line.split("//")[0].strip())
    return out


def test_products_wait_for_their_last_fetches(tmp_path):
    seen = 0
    for name, lines in assembly("muon_kernels.hip", tmp_path).items():
        if not re.search(r"ns_(product|last)I", name):
            continue
        fetch = [i for i, x in enumerate(lines) if x.startswith("buffer_load") and x.endswith(" lds")]
        after = next(i for i, x in enumerate(lines) if x.startswith("s_barrier") and i > fetch[-1])
        assert any(x.startswith("s_waitcnt") and "vmcnt(0)" in x for x in lines[fetch[-1]:after]), name
        seen += 1
    assert seen == 36, seen                          # 3 products and 3 types' last ones, 1 and 2 pieces, 3 tiles

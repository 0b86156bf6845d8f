"""The kernels of the built library as its own toolchain lists them: registers and instructions."""
import os
import re
import struct
import subprocess

LLVM = "/opt/rocm/llvm/bin"


def code_objects(library, folder):
    """Writes the gfx950 code objects bundled in the library into `folder`; returns their paths."""
    data = open(library, "rb").read()
    paths = []
    for m in re.finditer(rb"__CLANG_OFFLOAD_BUNDLE__", data):
        base = m.start()
        at = base + 24
        (n,) = struct.unpack_from("<Q", data, at)
        at += 8
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, at)
            name = data[at + 24:at + 24 + length]
            at += 24 + length
            if b"gfx950" in name and size:
                paths.append(os.path.join(folder, f"{len(paths)}.elf"))
                with open(paths[-1], "wb") as f:
                    f.write(data[base + offset:base + offset + size])
    return paths


def _tool(name, *args):
    return subprocess.run([os.path.join(LLVM, name), *args], check=True, text=True, stdout=subprocess.PIPE).stdout


def registers(paths):
    """{mangled kernel: (vector registers, vector spills)}."""
    got = {}
    for p in paths:
        for part in re.split(r"\n\s+- \.agpr_count:", _tool("llvm-readelf", "--notes", p))[1:]:
            name = re.search(r"\.name:\s+(\S+)\n(?:.*\n)*?\s+\.private_segment", part)[1]
            got[name] = tuple(int(re.search(rf"\.{f}:\s+(\d+)", part)[1]) for f in ("vgpr_count", "vgpr_spill_count"))
    return got


def instructions(path, pattern):
    """{mangled kernel: [instruction]} of the kernels that match, labels as lines that end in a colon."""
    got, lines = {}, None
    for line in _tool("llvm-objdump", "-d", "--no-show-raw-insn", "--no-leading-addr", path).splitlines():
        m = re.match(r"(?:[0-9a-f]+ )?<(\S+)>:", line)
        if m and not m[1].startswith("L"):
            lines = got.setdefault(m[1], []) if re.search(pattern, m[1]) else None
        elif m and lines is not None:
            lines.append(m[1] + ":")
        elif lines is not None and line.strip():
            lines.append(line.split("//")[0].strip())
    return got

"""The gfx950 code of the built library as text: the code objects in libmoe_get.so, disassembled."""
import os
import re
import struct
import subprocess
import tempfile

import combine_moe_get_amd as mg

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(lib=mg.LIB_PATH):
    """The gfx950 ELF images of a library's offload bundles."""
    data = open(lib, "rb").read()
    for m in re.finditer(re.escape(MAGIC), data):
        at = m.end()
        n, = struct.unpack_from("<Q", data, at)
        at += 8
        if n > 16:  # the text of a program, not a bundle
            continue
        for _ in range(n):
            off, size, tl = struct.unpack_from("<QQQ", data, at)
            triple = data[at + 24:at + 24 + tl]
            at += 24 + tl
            if b"gfx950" in triple and size:
                yield data[m.start() + off:m.start() + off + size]


def kernels(lib=mg.LIB_PATH):
    """{demangled kernel: its instructions in order}; a label is a line that ends with a colon."""
    found = {}
    for image in code_objects(lib):
        with tempfile.NamedTemporaryFile(suffix=".elf") as f:
            f.write(image)
            f.flush()
            text = subprocess.run([OBJDUMP, "-d", "-C", "--no-show-raw-insn", "--no-leading-addr", "--symbolize-operands",
                                   f.name], check=True, capture_output=True, text=True).stdout
        name = None
        for line in text.splitlines():
            line = line.split("//")[0].strip()
            m = re.fullmatch(r"(?:[0-9a-f]+ )?<(.*)>:", line)
            if m and not re.fullmatch(r"L\d+", m.group(1)):
                name = m.group(1)
                found[name] = []
            elif name is not None and line:
                found[name].append(m.group(1) + ":" if m else line)
    return found

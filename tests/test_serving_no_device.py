"""The windowed, 8-bit and rotating-append calls where no CUDA device can be
reached: valid arguments come back as PA_ERR_CUDA, whatever the sizes.  They
run in a process that sees no device, on host buffers that nothing reads."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALLS = ("pa_cache_append_i8", "pa_rope_append", "pa_rope_append_i8", "pa_decode_window", "pa_decode_i8",
         "pa_prefill_window", "pa_prefill_i8")

PROGRAM = """
import ctypes, sys
from paged_kv_attention_36_b200 import binding as pa

vp = ctypes.c_void_p
room = ctypes.create_string_buffer(1 << 16)
at = (ctypes.addressof(room) + 255) // 256 * 256
p = lambda i: vp(at + 4096 * i)  # noqa: E731
dims = pa.pa_dims(2, 8, 2, 64, 16, 4, 2)
d = ctypes.byref(dims)
rope = pa.pa_rope(at + 4096 * 7, at + 4096 * 8, 10, 64, 0)
for what in sys.argv[1:]:
    fn, scales = getattr(pa.lib, what), [p(5), p(6)] if what.endswith("i8") else []
    for n in (1, 3, 4000):  # tokens, or the longest sequence's queries
        if what == "pa_cache_append_i8":
            args = [p(0), p(1), p(2), n, p(3), p(4), *scales, d]
        elif "append" in what:
            args = [p(9), 512, p(0), 128, p(1), 128, ctypes.byref(rope), p(2), n, vp(at + (1 << 30)), p(3), p(4),
                    *scales, d]
        else:
            many, work = ([p(7), n], []) if "prefill" in what else ([], [p(10), 1 << 40])
            args = [p(0), *many, p(1), p(2), *scales, p(3), p(4), 0.1, 64, 4, p(8), d, *work]
        print(what, n, flush=True)
        print(fn(*args, None), flush=True)
"""


def test_no_device_is_an_error():
    r = subprocess.run([sys.executable, "-c", PROGRAM, *CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT))
    lines = r.stdout.splitlines()
    assert r.returncode == 0, f"ended with {r.returncode} in {lines[-1:]}: {r.stderr[-500:]}"
    assert dict(zip(lines[::2], lines[1::2])) == {f"{c} {n}": "-6" for c in CALLS for n in (1, 3, 4000)}

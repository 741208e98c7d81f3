"""The host code of the attention-side entry points under AddressSanitizer and
UndefinedBehaviorSanitizer (tests/attn_sanitize_driver.cpp): every size at the
ends of its type, on the CPU.  Built like tests/test_abi_sanitizers.py."""
import concurrent.futures
import os
import subprocess
import tempfile

import pytest

from test_abi_sanitizers import HERE, HIPCC, ROOT, SAN


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="no hipcc")
def test_attention_host_code_under_sanitizers():
    from sparse_linear_layers_group_amd import build as B
    csrc = os.path.join(ROOT, "sparse_linear_layers_group_amd", "csrc")
    with tempfile.TemporaryDirectory() as d:
        def run(*args, **kw):
            r = subprocess.run(args, capture_output=True, text=True, **kw)
            assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
            return r

        def comp(src):
            obj = os.path.join(d, os.path.basename(src) + ".o")
            run(HIPCC, *B.CFLAGS, *SAN, "-g", "-c", src, "-o", obj)
            return obj
        with concurrent.futures.ThreadPoolExecutor(4) as ex:
            objs = list(ex.map(comp, [os.path.join(csrc, f) for f in B.SOURCES] +
                               [os.path.join(HERE, "attn_sanitize_driver.cpp")]))
        exe = os.path.join(d, "attn_sanitized")
        run(HIPCC, "--offload-arch=gfx950", *SAN, *objs, "-o", exe)
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0",
                   UBSAN_OPTIONS="print_stacktrace=1", HIP_VISIBLE_DEVICES="")
        r = run(exe, env=env, timeout=300)
        assert "runtime error" not in r.stdout + r.stderr and "ran clean" in r.stdout

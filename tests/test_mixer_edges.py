"""The token-mixer operators on the host: what the compiled code assumes, and the limits of what a call accepts."""
import re
import subprocess

from convolution_forward_amd import build


def test_conv_promises_no_more_alignment_than_is_checked(tmp_path):
    """The four-channel bf16 form is chosen for 8-byte alignment: no global load or store of it may assume more."""
    out = tmp_path / "conv.ll"
    subprocess.run([build.HIPCC, *build.COMMON_FLAGS, "--offload-device-only", "-S", "-emit-llvm",
                    build.CSRC + "/causal_conv1d.hip", "-o", str(out)], check=True, capture_output=True)
    seen = 0
    for body in re.findall(r"^define .*?^}", out.read_text(), re.S | re.M):
        form = re.search(r"causal_conv1d_kernelI(\w)Li(\d)ELi\dE", body)
        if not form:
            continue
        most = int(form[2]) * {"t": 2, "f": 4}[form[1]]
        aligned = [int(a) for a in re.findall(r"(?:load|store) .*?addrspace\(1\).*?align (\d+)", body)]
        assert aligned and max(aligned) <= max(most, 4), form[0]    # (biases and offsets are 4-byte values)
        seen += 1
    assert seen == 28       # two types, two widths, 2 to 8 taps

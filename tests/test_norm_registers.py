"""The norm keeps a row's values in registers between the sum of squares and the encode. The compiler's own
report says whether it does: an instance whose registers do not suffice moves values through memory."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rows_of_whole_waves_stay_in_registers(tmp_path):
    from fp8_group_quant_amd import build
    src = os.path.join(build.CSRC, "norm.hip")
    r = subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-c", src, "-o", str(tmp_path / "norm.o"),
                        "-Rpass-analysis=kernel-resource-usage"], capture_output=True, text=True, check=True)
    scratch = dict(re.findall(r"Function Name: (\S+).*?ScratchSize \[bytes/lane\]: (\d+)", r.stderr, re.S))
    whole = {n: int(b) for n, b in scratch.items() if re.search(r"rms_norm_quant_kernelILi\dELi64E", n)}
    assert len(whole) == 21  # three types, seven lengths
    assert not any(whole.values()), whole
